// kvpages.cu -- the bookkeeping of the paged key/value cache, on the GPU:
// block tables, slot maps and the stack of free pages, from request lengths.
//
//   truncate  request b keeps keep_b of its len_b tokens; the pages behind
//             them go back on the stack and their table entries become -1.
//             Of the n pages freed (request order, then block order) the i-th
//             lands at stack[count + n - 1 - i].  An entry that is -1 already (a
//             page given back before) frees none: the scan counts entries as it
//             finds them, not as lengths make them.
//   extend    request b gets new_b tokens: pages for blocks ceil(len_b / P) ..
//             ceil((len_b + new_b) / P) - 1 -- the i-th handed out (request
//             order) is stack[count - 1 - i] -- and for each new token its
//             slot, page * P + offset.
// Taking pages in the order in which truncate left them on top makes extend
// its exact inverse: drafted tokens that are dropped and replaced by as many
// find the same pages again.
//
// A few KB in, a slot (8 bytes) per token out: the launch and a chain of
// dependent reads bound it, not bandwidth.  So each is one launch with no
// scratch memory and no atomics on global memory.
//   extend    every CTA scans all requests for itself (two integer prefix sums
//             over B lengths read from L2), and only the filling of tables and
//             slots is divided.  A page id is read once per 32 blocks and passed
//             on by shuffles.  Where an output overwrites an input, the CTAs are
//             one cluster (of at most eight, the portable limit) with its
//             barrier between the last read of an input and the first write
//             of an output; otherwise there are as many as the slots keep busy.
//   truncate  the table is an input that is always overwritten, and pages must be
//             counted as they are found, so the CTAs of a cluster share the
//             requests out, and read each other's totals.
// Measured, truncate and extend together: 64 requests 7.2 us; 2048 requests, a
// tenth of them with whole prompts (200000 new tokens), 16.4 us (with a page
// read per token and eight CTAs 39; with truncate's pages taken from the lengths,
// holes and all, 14.5; with every one of its CTAs counting all rows 27).
#include <atomic>
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
constexpr int PG_MAX_REQUESTS = 16384;
constexpr int PG_SMEM_FREE = 48 * 1024;     // shared memory that a launch gets unasked

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

// Rows that lose up to PG_SHORT blocks (dropped drafts) are looked after by a
// thread each, longer ones (finished requests) by a warp, with PG_BATCH loads of
// a lane on their way for each of PG_ROWS rows.
constexpr int PG_SHORT = 2;
constexpr int PG_BATCH = 4;
constexpr int PG_ROWS = 4;

// The requests of each of `ctas` CTAs.
__host__ __device__ __forceinline__ int pages_share(int requests, int ctas) {
  return (requests + ctas - 1) / ctas;
}

__global__ void __launch_bounds__(PG_THREADS) kv_truncate_kernel(const PagesArgs a) {
  // per request: first page freed, lengths before and after, a short row's entries
  extern __shared__ int sm_req[];
  __shared__ long long sm_scan[2 * PG_WARPS];
  __shared__ long long sm_total;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x, ctas = gridDim.x, share = pages_share(a.requests, ctas);
  const int first = min(a.requests, rank * share), B = min(share, a.requests - first);
  int* sm_rank = sm_req;
  int* sm_len = sm_rank + share;
  int* sm_keep = sm_len + share;
  int* sm_page = sm_keep + share;           // [PG_SHORT][share]
  const int per = (B + PG_THREADS - 1) / PG_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long count = *a.count;
  count = count < 0 ? 0 : (count > a.stack_size ? a.stack_size : count);
  auto blocks_in_row = [&](long long tokens) {
    const long long n = blocks_of(tokens < 0 ? 0 : tokens, a.page_shift);
    return n < a.width ? n : a.width;
  };
  auto row_of = [&](int b) { return a.table + static_cast<long long>(first + b) * a.table_stride; };
  // the blocks that a request loses: from j0 on
  auto blocks = [&](int b, long long& j0) {
    j0 = blocks_in_row(sm_keep[b]);
    return static_cast<int>(blocks_in_row(sm_len[b]) - j0);
  };
  // The pages among them, per request.  Short rows: each thread for its own.
  for (int b = b0; b < b1; ++b) {
    const int len = a.lens[first + b], keep = max(0, min(a.change[first + b], len));
    sm_len[b] = len;
    sm_keep[b] = len < 0 ? len : keep;
    long long j0;
    const int n = blocks(b, j0);
    int pages = 0;
    if (n <= PG_SHORT) {
#pragma unroll
      for (int i = 0; i < PG_SHORT; ++i) {
        const int page = i < n ? row_of(b)[j0 + i] : -1;
        sm_page[i * share + b] = page;
        pages += page >= 0;
      }
    }
    sm_rank[b] = n <= PG_SHORT ? pages : -1;
  }
  __syncthreads();
  // Long ones: a warp looks after the requests whose number is its own modulo the
  // warps, so that neighbours (which often end together) go to different ones.
  auto each_long = [&](auto f) {
    for (int base = warp; base < B; base += 32 * PG_WARPS) {
      const int mine = base + lane * PG_WARPS;
      long long j0;
      uint32_t bits = __ballot_sync(0xFFFFFFFFu, mine < B && blocks(mine, j0) > PG_SHORT);
      f(base, bits);
    }
  };
  each_long([&](int base, uint32_t bits) {
    while (bits) {
      int b[PG_ROWS], n[PG_ROWS], pages[PG_ROWS], most = 0;
      long long j0[PG_ROWS];
#pragma unroll
      for (int u = 0; u < PG_ROWS; ++u) {
        n[u] = pages[u] = 0;
        b[u] = -1;
        if (bits) {
          b[u] = base + (__ffs(bits) - 1) * PG_WARPS;
          bits &= bits - 1;
          n[u] = blocks(b[u], j0[u]);
        }
        most = max(most, n[u]);
      }
      for (int k = lane; k < most; k += 32 * PG_BATCH) {
        int page[PG_ROWS][PG_BATCH];
#pragma unroll
        for (int u = 0; u < PG_ROWS; ++u)
#pragma unroll
          for (int i = 0; i < PG_BATCH; ++i)
            page[u][i] = k + 32 * i < n[u] ? row_of(b[u])[j0[u] + k + 32 * i] : -1;
#pragma unroll
        for (int u = 0; u < PG_ROWS; ++u)
#pragma unroll
          for (int i = 0; i < PG_BATCH; ++i) pages[u] += page[u][i] >= 0;
      }
#pragma unroll
      for (int u = 0; u < PG_ROWS; ++u) {
        const int all = __reduce_add_sync(0xFFFFFFFFu, pages[u]);
        if (lane == 0 && b[u] >= 0) sm_rank[b[u]] = all;
      }
    }
  });
  __syncthreads();
  Pair mine{0, 0}, all;
  for (int b = b0; b < b1; ++b) mine.a += sm_rank[b];
  Pair at = block_scan(mine, sm_scan, all);
  for (int b = b0; b < b1; ++b) {
    const int n = sm_rank[b];
    sm_rank[b] = static_cast<int>(at.a);
    at.a += n;
  }
  long long total = all.a, before = 0;
  if (ctas > 1) {
    if (tid == 0) sm_total = all.a;
    cluster_sync();                         // every CTA has read its inputs and counted its pages
    total = lane < ctas ? ld_shared_cluster_s64(map_to_cta(smem_u32(&sm_total), lane)) : 0;
    before = lane < rank ? total : 0;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      total += __shfl_xor_sync(0xFFFFFFFFu, total, d);
      before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
    }
    cluster_arrive();
  } else {
    __syncthreads();
  }
  for (int b = tid; b < B; b += PG_THREADS) a.lens_out[first + b] = sm_keep[b];
  if (rank == 0 && tid == 0) {
    const long long n = count + total;
    a.counts_out[0] = static_cast<int>(n < a.stack_size ? n : a.stack_size);
    a.counts_out[1] = static_cast<int>(n < a.stack_size ? 0 : n - a.stack_size);
  }
  const long long top = count + total - 1 - before;
  auto push = [&](int page, int i) {
    if (top - i < a.stack_size) a.stack[top - i] = page;
  };
  for (int b = tid; b < B; b += PG_THREADS) {
    long long j0;
    const int n = blocks(b, j0);
    if (n > PG_SHORT) continue;
    int i_th = sm_rank[b];
#pragma unroll
    for (int i = 0; i < PG_SHORT; ++i) {
      const int page = sm_page[i * share + b];
      if (page >= 0) {
        push(page, i_th++);
        row_of(b)[j0 + i] = -1;
      }
    }
  }
  each_long([&](int base, uint32_t bits) {
    for (; bits; bits &= bits - 1) {
      const int b = base + (__ffs(bits) - 1) * PG_WARPS;
      long long j0;
      const int n = blocks(b, j0);
      int i_th = sm_rank[b];
      int* row = row_of(b) + j0;
      for (int k0 = 0; k0 < n; k0 += 32 * PG_BATCH) {
        const int k = k0 + lane;
        int page[PG_BATCH];
#pragma unroll
        for (int i = 0; i < PG_BATCH; ++i) page[i] = k + 32 * i < n ? row[k + 32 * i] : -1;
#pragma unroll
        for (int i = 0; i < PG_BATCH; ++i) {
          const uint32_t have = __ballot_sync(0xFFFFFFFFu, page[i] >= 0);
          if (page[i] >= 0) {
            push(page[i], i_th + __popc(have & ((1u << lane) - 1u)));
            row[k + 32 * i] = -1;
          }
          i_th += __popc(have);
        }
      }
    }
  });
  __syncwarp();
  if (ctas > 1) cluster_wait();             // nobody reads this CTA's total any more
}

cudaError_t launch_pages(void (*kern)(const PagesArgs), const PagesArgs& a, int64_t ctas,
                         size_t smem, cudaStream_t st) {
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
  const char* in[3] = {reinterpret_cast<const char*>(lens), reinterpret_cast<const char*>(fresh),
                       reinterpret_cast<const char*>(count)};
  const int64_t in_bytes[3] = {4 * requests, 4 * requests, 4};
  const char* out[3] = {reinterpret_cast<const char*>(lens_out),
                        reinterpret_cast<const char*>(counts_out), reinterpret_cast<const char*>(cu)};
  const int64_t out_bytes[3] = {4 * requests, 8, 4 * (requests + 1)};
  for (int i = 0; i < 3; ++i)
    for (int o = 0; o < 3; ++o)
      if (in[i] < out[o] + out_bytes[o] && out[o] < in[i] + in_bytes[i]) a.in_place = 1;
  // a warp for every 4 requests or 128 slots
  const int64_t want = (requests / 4 + max_tokens / 128) / PG_WARPS;
  const int64_t most = a.in_place ? PG_CLUSTER : PG_MAX_CTAS;
  const int64_t ctas = want < 1 ? 1 : (want > most || a.in_place ? most : want);
  const size_t smem = (3 * requests + 1) * sizeof(int);
  if (smem > PG_SMEM_FREE) {
    // the limit belongs to the kernel, not to the launch: once, to the most that
    // any call needs, so that calls on several host threads leave each other theirs
    constexpr int most_smem = (3 * PG_MAX_REQUESTS + 1) * sizeof(int);
    static std::atomic<bool> set[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
      e = cudaFuncSetAttribute(kv_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
      if (e != cudaSuccess) return e;
      if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
    }
  }
  return launch_pages(kv_extend_kernel, a, ctas, smem, st);
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
  a.in_place = 1;                           // the table
  // one CTA where its threads have a request each: a cluster's barriers take
  // longer than sharing out saves
  const int ctas = requests <= PG_THREADS ? 1 : PG_CLUSTER;
  static_assert((3 + PG_SHORT) * PG_MAX_REQUESTS / PG_CLUSTER * sizeof(int) <= PG_SMEM_FREE, "");
  return launch_pages(kv_truncate_kernel, a, ctas, (3 + PG_SHORT) * pages_share(a.requests, ctas) * sizeof(int), st);
}

}  // namespace mxk
