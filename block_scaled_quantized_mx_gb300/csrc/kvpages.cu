// kvpages.cu -- the bookkeeping of the paged key/value cache, on the GPU:
// block tables, slot maps and the stack of free pages, from request lengths.
//
//   truncate  request b keeps keep_b of its len_b tokens; the pages behind
//             them go back on the stack and their table entries become -1.
//             Of the n pages freed (request order, then block order) the i-th
//             lands at stack[count + n - 1 - i].
//   extend    request b gets new_b tokens: pages for blocks ceil(len_b / P) ..
//             ceil((len_b + new_b) / P) - 1 -- the i-th handed out (request
//             order) is stack[count - 1 - i] -- and for each new token its
//             slot, page * P + offset.
// Taking pages in the order in which truncate left them on top makes extend
// its exact inverse: drafted tokens that are dropped and replaced by as many
// find the same pages again.
//
// A few KB in, a slot (8 bytes) per token out: the launch and a chain of
// dependent reads bound it, not bandwidth.  So it is one launch with no
// scratch memory and no atomics on global memory: every CTA scans all
// requests for itself (two integer prefix sums over B lengths read from L2),
// and only the filling of tables and slots is divided.  A page id is read
// once per 32 blocks and passed on by shuffles.  Where an output overwrites an
// input, the CTAs are one cluster (of at most eight, the portable limit) with
// its barrier between the last read of an input and the first write of an
// output; otherwise there are as many as the slots keep busy.
// Measured, truncate and extend together: 64 requests 7.4 us; 2048 requests, a
// tenth of them with whole prompts (200000 new tokens), 14.7 us (with a page
// read per token and eight CTAs 39).
#include <cstdint>

#include "common.cuh"
#include "kv_common.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int PG_THREADS = 512;
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_CLUSTER = 8;
constexpr int PG_MAX_CTAS = 128;

// Sum of two values over the block's threads before this one (exclusive), in
// thread order; `all` receives the block's totals.  Uses `sm` (2 x PG_WARPS).
struct Pair {
  long long a, b;
};
__device__ __forceinline__ Pair block_scan(Pair v, long long* sm, Pair& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Pair s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long ua = __shfl_up_sync(0xFFFFFFFFu, s.a, d);
    const long long ub = __shfl_up_sync(0xFFFFFFFFu, s.b, d);
    if (lane >= d) {
      s.a += ua;
      s.b += ub;
    }
  }
  if (lane == 31) {
    sm[2 * warp] = s.a;
    sm[2 * warp + 1] = s.b;
  }
  __syncthreads();
  // every warp scans the warps' totals for itself
  static_assert(PG_WARPS <= 32, "one total per lane");
  Pair t{lane < PG_WARPS ? sm[2 * lane] : 0, lane < PG_WARPS ? sm[2 * lane + 1] : 0};
#pragma unroll
  for (int d = 1; d < PG_WARPS; d <<= 1) {
    const long long ua = __shfl_up_sync(0xFFFFFFFFu, t.a, d);
    const long long ub = __shfl_up_sync(0xFFFFFFFFu, t.b, d);
    if (lane >= d) {
      t.a += ua;
      t.b += ub;
    }
  }
  all.a = __shfl_sync(0xFFFFFFFFu, t.a, PG_WARPS - 1);
  all.b = __shfl_sync(0xFFFFFFFFu, t.b, PG_WARPS - 1);
  const long long ba = __shfl_sync(0xFFFFFFFFu, t.a, warp ? warp - 1 : 0);
  const long long bb = __shfl_sync(0xFFFFFFFFu, t.b, warp ? warp - 1 : 0);
  return Pair{(warp ? ba : 0) + s.a - v.a, (warp ? bb : 0) + s.b - v.b};
}

struct PagesArgs {
  const int* lens;
  const int* change;        // extend: new tokens; truncate: tokens kept
  int* table;
  long long table_stride;
  long long width;
  int* stack;
  long long stack_size;
  const int* count;
  int page_shift;
  int requests;
  int* lens_out;
  int* cu;
  long long* slots;
  long long max_tokens;
  int* counts_out;
  int in_place;             // an output overwrites an input: the CTAs are a cluster
};

__device__ __forceinline__ long long blocks_of(long long tokens, int shift) {
  return (tokens + (1ll << shift) - 1) >> shift;
}

__global__ void __launch_bounds__(PG_THREADS) kv_extend_kernel(const PagesArgs a) {
  extern __shared__ int sm_req[];           // per request: first token, first page, length
  __shared__ long long sm_scan[2 * PG_WARPS];
  __shared__ int sm_cut, sm_served;
  __shared__ long long sm_total[2];
  const int B = a.requests, tid = threadIdx.x;
  int* sm_cu = sm_req;                      // B + 1
  int* sm_rank = sm_cu + B + 1;             // B
  int* sm_len = sm_rank + B;                // B
  const int per = (B + PG_THREADS - 1) / PG_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long avail = *a.count;
  avail = avail < 0 ? 0 : (avail > a.stack_size ? a.stack_size : avail);
  const long long capacity = a.width << a.page_shift;
  if (tid == 0) {
    sm_cut = B;
    sm_served = 0;
  }
  // Each request's need and new tokens, kept in the arrays that later hold its
  // first page and first token; -1 new tokens for a request that is refused
  // on its own: a negative length or count, or more tokens than a table row
  // holds.
  Pair mine{0, 0}, all;
  for (int b = b0; b < b1; ++b) {
    const int len = a.lens[b];
    const long long fresh = a.change[b];
    const bool ok = len >= 0 && fresh >= 0 && len + fresh <= capacity && len + fresh <= 0x7FFFFFFF;
    const long long need =
        ok ? blocks_of(len + fresh, a.page_shift) - blocks_of(len, a.page_shift) : 0;
    sm_len[b] = len;
    sm_cu[b] = ok ? static_cast<int>(fresh) : -1;
    sm_rank[b] = static_cast<int>(need);
    mine.a += need;
    mine.b += ok ? fresh : 0;
  }
  const Pair at = block_scan(mine, sm_scan, all);
  if (tid == 0) {
    sm_total[0] = all.a;
    sm_total[1] = all.b;
  }
  // the first request that does not fit; it and all behind it are refused
  {
    Pair p = at;
    for (int b = b0; b < b1; ++b) {
      p.a += sm_rank[b];
      p.b += max(0, sm_cu[b]);
      if (p.a > avail || p.b > a.max_tokens) {
        atomicMin(&sm_cut, b);
        break;
      }
    }
  }
  __syncthreads();
  const int cut = sm_cut;
  {
    Pair p = at;
    int served = 0;
    for (int b = b0; b < b1; ++b) {
      const int need = sm_rank[b], fresh = sm_cu[b];
      if (b == cut) {
        sm_total[0] = p.a;
        sm_total[1] = p.b;
      }
      sm_cu[b] = b <= cut ? static_cast<int>(p.b) : -1;   // -1: the total, filled in below
      sm_rank[b] = static_cast<int>(b <= cut ? p.a : 0);
      p.a += need;
      p.b += max(0, fresh);
      served += fresh >= 0 && b < cut;
    }
    if (served) atomicAdd(&sm_served, served);
  }
  __syncthreads();
  const int total_pages = static_cast<int>(sm_total[0]);
  const int total = static_cast<int>(sm_total[1]);
  for (int b = b0; b < b1; ++b)
    if (b > cut) sm_cu[b] = total;
  if (tid == 0) sm_cu[B] = total;
  __syncthreads();
  if (a.in_place) cluster_sync();           // every CTA has read its inputs
  const int rank = blockIdx.x, ctas = gridDim.x;
  for (int b = rank * PG_THREADS + tid; b <= B; b += ctas * PG_THREADS) {
    a.cu[b] = sm_cu[b];
    if (b < B) a.lens_out[b] = sm_len[b] + (sm_cu[b + 1] - sm_cu[b]);
  }
  if (rank == 0 && tid == 0) {
    a.counts_out[0] = static_cast<int>(avail) - total_pages;
    a.counts_out[1] = B - sm_served;
  }
  // one warp per request fills its row of the table and its slots
  const int warp = tid >> 5, lane = tid & 31;
  const int P = 1 << a.page_shift;
  for (int b = rank * PG_WARPS + warp; b < B; b += ctas * PG_WARPS) {
    const int first = sm_cu[b], n = sm_cu[b + 1] - first, len = sm_len[b];
    if (n == 0) continue;
    int* row = a.table + static_cast<long long>(b) * a.table_stride;
    const long long had = blocks_of(len, a.page_shift);
    const long long has = blocks_of(static_cast<long long>(len) + n, a.page_shift);
    const int* top = a.stack + (avail - 1 - sm_rank[b]);
    // 32 blocks at a time, a page id per lane: a partly filled last block's
    // from the table, new ones from the stack (one load for up to 32 P tokens)
    const long long end = static_cast<long long>(len) + n;
    for (long long j0 = len >> a.page_shift; j0 < has; j0 += 32) {
      const long long j = j0 + lane;
      int page = -1;
      if (j < had) {
        page = row[j];
      } else if (j < has) {
        page = top[had - j];
        row[j] = page;
      }
      const long long p0 = j0 << a.page_shift;
      const long long from = p0 > len ? p0 : len;
      const long long to = min(end, p0 + (32ll << a.page_shift));
      for (long long t = from; t < to; t += 32) {
        const long long pos = t + lane;
        const int id = __shfl_sync(0xFFFFFFFFu, page,
                                   static_cast<int>((pos >> a.page_shift) - j0) & 31);
        if (pos < to)
          a.slots[first + (pos - len)] = static_cast<long long>(id) * P + (pos & (P - 1));
      }
    }
  }
  for (long long t = total + rank * PG_THREADS + tid; t < a.max_tokens; t += ctas * PG_THREADS)
    a.slots[t] = -1;
}

__global__ void __launch_bounds__(PG_THREADS) kv_truncate_kernel(const PagesArgs a) {
  extern __shared__ int sm_req[];           // per request: first page freed, lengths before and after
  __shared__ long long sm_scan[2 * PG_WARPS];
  const int B = a.requests, tid = threadIdx.x;
  int* sm_rank = sm_req;
  int* sm_len = sm_rank + B;
  int* sm_keep = sm_len + B;
  const int per = (B + PG_THREADS - 1) / PG_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long count = *a.count;
  count = count < 0 ? 0 : (count > a.stack_size ? a.stack_size : count);
  auto blocks_in_row = [&](long long tokens) {
    const long long n = blocks_of(tokens < 0 ? 0 : tokens, a.page_shift);
    return n < a.width ? n : a.width;
  };
  Pair mine{0, 0}, all;
  for (int b = b0; b < b1; ++b) {
    const int len = a.lens[b], keep = max(0, min(a.change[b], len));
    sm_len[b] = len;
    sm_keep[b] = len < 0 ? len : keep;
    mine.a += blocks_in_row(len) - blocks_in_row(keep);
  }
  Pair at = block_scan(mine, sm_scan, all);
  for (int b = b0; b < b1; ++b) {
    sm_rank[b] = static_cast<int>(at.a);
    at.a += blocks_in_row(sm_len[b]) - blocks_in_row(sm_keep[b]);
  }
  __syncthreads();
  if (a.in_place) cluster_sync();           // every CTA has read its inputs
  const int rank = blockIdx.x, ctas = gridDim.x;
  for (int b = rank * PG_THREADS + tid; b < B; b += ctas * PG_THREADS) a.lens_out[b] = sm_keep[b];
  if (rank == 0 && tid == 0) {
    const long long n = count + all.a;
    a.counts_out[0] = static_cast<int>(n < a.stack_size ? n : a.stack_size);
    a.counts_out[1] = static_cast<int>(n < a.stack_size ? 0 : n - a.stack_size);
  }
  const int warp = tid >> 5, lane = tid & 31;
  for (int b = rank * PG_WARPS + warp; b < B; b += ctas * PG_WARPS) {
    const long long j0 = blocks_in_row(sm_keep[b]), j1 = blocks_in_row(sm_len[b]);
    int* row = a.table + static_cast<long long>(b) * a.table_stride;
    for (long long j = j0 + lane; j < j1; j += 32) {
      const long long to = count + all.a - 1 - (sm_rank[b] + (j - j0));
      if (to < a.stack_size) a.stack[to] = row[j];
      row[j] = -1;
    }
  }
}

cudaError_t launch_pages(void (*kern)(const PagesArgs), PagesArgs& a, size_t smem,
                         cudaStream_t st) {
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  const char* in[3] = {reinterpret_cast<const char*>(a.lens),
                       reinterpret_cast<const char*>(a.change),
                       reinterpret_cast<const char*>(a.count)};
  const int64_t in_bytes[3] = {4ll * a.requests, 4ll * a.requests, 4};
  const char* out[3] = {reinterpret_cast<const char*>(a.lens_out),
                        reinterpret_cast<const char*>(a.counts_out),
                        reinterpret_cast<const char*>(a.cu)};
  const int64_t out_bytes[3] = {4ll * a.requests, 8, a.cu ? 4ll * (a.requests + 1) : 0};
  a.in_place = 0;
  for (int i = 0; i < 3; ++i)
    for (int o = 0; o < 3; ++o)
      if (in[i] < out[o] + out_bytes[o] && out[o] < in[i] + in_bytes[i]) a.in_place = 1;
  // a warp for every 4 requests or 128 slots
  const int64_t want = (a.requests / 4 + a.max_tokens / 128) / PG_WARPS;
  const int64_t most = a.in_place ? PG_CLUSTER : PG_MAX_CTAS;
  const int64_t ctas = want < 1 ? 1 : (want > most ? most : (a.in_place ? PG_CLUSTER : want));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(PG_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.in_place ? static_cast<unsigned>(ctas) : 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_kv_extend(const int* lens, const int* fresh, int64_t requests, int* table,
                             int64_t table_stride, int64_t width, const int* stack,
                             int64_t stack_size, const int* count, int page, int* lens_out,
                             int* cu, int64_t* slots, int64_t max_tokens, int* counts_out,
                             cudaStream_t st) {
  PagesArgs a{};
  a.lens = lens;
  a.change = fresh;
  a.table = table;
  a.table_stride = table_stride;
  a.width = width;
  a.stack = const_cast<int*>(stack);        // extend only reads it
  a.stack_size = stack_size;
  a.count = count;
  a.page_shift = kv_page_shift(page);
  a.requests = static_cast<int>(requests);
  a.lens_out = lens_out;
  a.cu = cu;
  a.slots = reinterpret_cast<long long*>(slots);
  a.max_tokens = max_tokens;
  a.counts_out = counts_out;
  return launch_pages(kv_extend_kernel, a, (3 * requests + 1) * sizeof(int), st);
}

cudaError_t launch_kv_truncate(const int* lens, const int* keep, int64_t requests, int* table,
                               int64_t table_stride, int64_t width, int* stack,
                               int64_t stack_size, const int* count, int page, int* lens_out,
                               int* counts_out, cudaStream_t st) {
  PagesArgs a{};
  a.lens = lens;
  a.change = keep;
  a.table = table;
  a.table_stride = table_stride;
  a.width = width;
  a.stack = stack;
  a.stack_size = stack_size;
  a.count = count;
  a.page_shift = kv_page_shift(page);
  a.requests = static_cast<int>(requests);
  a.lens_out = lens_out;
  a.counts_out = counts_out;
  return launch_pages(kv_truncate_kernel, a, 3 * requests * sizeof(int), st);
}

}  // namespace mxk
