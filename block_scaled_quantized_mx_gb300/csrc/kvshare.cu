// kvshare.cu -- pages of the paged cache that several requests hold.
//
// refs[p] counts page p's holders beyond the first: 0 for a free page and for one
// that a single request holds, as every page is that extend hands out.
//   fork     request dst_i becomes the first keep_i tokens of request src_i and holds
//            the same pages, the last, partly filled one among them
//   own      a request that is about to write its partly filled last page, which
//            others hold too, gets a copy of it on a page from the stack; where all of
//            a page's holders are about to, the last of them keeps the page
//   release  truncate for shared pages: a page goes on the stack when its last
//            holder lets it go, and counts as freed by the last of the requests (in
//            their order) that do so in one call
// fork and release move a few KB and own's plan less: launches and chains of
// dependent reads bound them, HBM own's copies (L2, where several requests copy one
// page).
// Measured, release + fork + own with its copies: 16 samples of a prompt of 1000 tokens 19 us;
// eight samples of each of 64 prompts of up to 4096 tokens 36 us, about 13, 5, 7 and 10 of
// them.  (release with eight lanes a row and its entries read again in each step took 27, with
// every dropped page's holder settled by an atomic 18.)
//
// Who is the last of several holders must not hang on the order of atomics.  So
// counts go down first; a page whose count is then negative has lost its last holder, and
// those who let it go bid with atomicMin(-2 - request) for it: the count itself holds
// the bids, the largest request wins, and sets it to 0.  Barriers between the steps:
// the CTAs are one cluster.
#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "kv_common.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int SH_THREADS = 1024;
constexpr int SH_WARPS = SH_THREADS / 32;
constexpr int SH_CLUSTER = 8, SH_WIDE = 16; // CTAs, where there are many requests
constexpr int SH_MAX_REQUESTS = 16384;
constexpr int SH_ROWS = 4;                  // requests that a warp looks after together,
constexpr int SH_BATCH = 2;                 // with as many table entries of each a lane
constexpr int SH_SPAN = 32 * SH_BATCH;      // entries of a row at once
constexpr int SH_SMEM_FREE = 48 * 1024;     // shared memory that a launch gets unasked

struct ShareArgs {
  const int* lens;
  const int* change;          // release: tokens kept; own: new tokens
  int* table;
  long long table_stride;
  long long width;
  int* stack;
  long long stack_size;
  const int* count;
  int* refs;
  int pages;
  int page_shift;
  int requests;
  const int* src;             // fork
  const int* dst;
  const int* keep;
  int forks;
  int* lens_out;              // own: the new tokens that are allowed
  int* copies;                // own
  int* counts_out;
};

// Sum over the block's threads before this one, in thread order, and of all.
__device__ __forceinline__ int share_scan(int v, int* sm, int& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += u;
  }
  if (lane == 31) sm[warp] = s;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < SH_WARPS; ++w) {
    if (w < warp) before += sm[w];
    all += sm[w];
  }
  return before + s - v;
}

__device__ __forceinline__ long long share_blocks(long long tokens, int shift, long long width) {
  const long long n = tokens <= 0 ? 0 : (tokens + (1ll << shift) - 1) >> shift;
  return n < width ? n : width;
}

// All of the grid (one cluster, or one CTA) has come here, and what it wrote is
// seen.
__device__ __forceinline__ void share_sync() {
  if (gridDim.x > 1)
    cluster_sync();
  else
    __syncthreads();
}

__host__ __device__ __forceinline__ int share_of(int requests, int ctas) {
  return (requests + ctas - 1) / ctas;
}

__global__ void __launch_bounds__(SH_THREADS) kv_release_kernel(const ShareArgs a) {
  extern __shared__ int sm_req[];           // per request: tokens before and after, pages freed
  __shared__ int sm_scan[SH_WARPS];
  __shared__ long long sm_total;
  wait_for_stream();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x, share = share_of(a.requests, ctas);
  const int first = min(a.requests, rank * share), B = min(share, a.requests - first);
  int* sm_len = sm_req;
  int* sm_keep = sm_len + share;
  int* sm_rank = sm_keep + share;
  long long count = *a.count;
  count = count < 0 ? 0 : (count > a.stack_size ? a.stack_size : count);
  for (int b = tid; b < B; b += SH_THREADS) {
    const int len = a.lens[first + b];
    sm_len[b] = len;
    sm_keep[b] = len < 0 ? len : max(0, min(a.change[first + b], len));
    sm_rank[b] = 0;
  }
  __syncthreads();
  // A warp's requests, SH_ROWS at a time, SH_SPAN entries of each, in page[][] (-1 behind a
  // row's last lost entry): f(the requests, their rows from the first of those entries).
  // Neighbours, which often end together, go to different warps.  Where that is all
  // that the warp has, the entries are read once and stay in registers over the steps.
  int page[SH_ROWS][SH_BATCH];
  bool kept = false;
  auto each = [&](auto f) {
    for (int base = warp; base < B; base += SH_WARPS * SH_ROWS) {
      int b[SH_ROWS], n[SH_ROWS], most = 0;
      int* row[SH_ROWS];
#pragma unroll
      for (int u = 0; u < SH_ROWS; ++u) {
        b[u] = base + u * SH_WARPS;
        n[u] = 0;
        row[u] = nullptr;
        if (b[u] < B) {
          const long long j0 = share_blocks(sm_keep[b[u]], a.page_shift, a.width);
          n[u] = static_cast<int>(share_blocks(sm_len[b[u]], a.page_shift, a.width) - j0);
          row[u] = a.table + static_cast<long long>(first + b[u]) * a.table_stride + j0;
        }
        most = max(most, n[u]);
      }
      const bool all = B <= SH_WARPS * SH_ROWS && most <= SH_SPAN;
      for (int k0 = 0; k0 < most; k0 += SH_SPAN) {
        if (!(all && kept)) {
#pragma unroll
          for (int u = 0; u < SH_ROWS; ++u)
#pragma unroll
            for (int i = 0; i < SH_BATCH; ++i) {
              const int k = 32 * i + lane;   // (row[u] has moved on by k0)
              page[u][i] = k0 + k < n[u] ? row[u][k] : -1;
            }
        }
        f(b, row);
#pragma unroll
        for (int u = 0; u < SH_ROWS; ++u) row[u] += SH_SPAN;
      }
      kept = true;
    }
  };
  auto held = [&](int p) { return p >= 0 && p < a.pages; };
  using Ints = int (&)[SH_ROWS];
  using Rows = int* (&)[SH_ROWS];
  each([&](Ints, Rows) {
#pragma unroll
    for (int u = 0; u < SH_ROWS; ++u)
#pragma unroll
      for (int i = 0; i < SH_BATCH; ++i)
        if (held(page[u][i])) atomicSub(a.refs + page[u][i], 1);
  });
  share_sync();
  each([&](Ints b, Rows row) {
    int refs[SH_ROWS][SH_BATCH];
#pragma unroll
    for (int u = 0; u < SH_ROWS; ++u)
#pragma unroll
      for (int i = 0; i < SH_BATCH; ++i)
        refs[u][i] = held(page[u][i]) ? __ldcg(a.refs + page[u][i]) : 0;
#pragma unroll
    for (int u = 0; u < SH_ROWS; ++u)
#pragma unroll
      for (int i = 0; i < SH_BATCH; ++i) {
        if (page[u][i] < 0) continue;
        if (refs[u][i] < 0) {
          atomicMin(a.refs + page[u][i], -2 - (first + b[u]));
        } else {
          row[u][32 * i + lane] = -1;       // others hold it (or it is none)
          page[u][i] = -1;
        }
      }
  });
  share_sync();
  each([&](Ints b, Rows row) {
    int was[SH_ROWS][SH_BATCH];
#pragma unroll
    for (int u = 0; u < SH_ROWS; ++u)
#pragma unroll
      for (int i = 0; i < SH_BATCH; ++i)
        was[u][i] = page[u][i] >= 0 ? atomicCAS(a.refs + page[u][i], -2 - (first + b[u]), 0) : 0;
#pragma unroll
    for (int u = 0; u < SH_ROWS; ++u) {
      int mine = 0;
#pragma unroll
      for (int i = 0; i < SH_BATCH; ++i) {
        if (page[u][i] < 0) continue;
        if (was[u][i] == -2 - (first + b[u])) {
          ++mine;
        } else {
          row[u][32 * i + lane] = -1;       // another request frees it
          page[u][i] = -1;
        }
      }
      mine = __reduce_add_sync(0xFFFFFFFFu, mine);
      if (lane == 0 && mine) sm_rank[b[u]] += mine;
    }
  });
  __syncthreads();
  const int per = (B + SH_THREADS - 1) / SH_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  int mine = 0, all;
  for (int b = b0; b < b1; ++b) mine += sm_rank[b];
  int at = share_scan(mine, sm_scan, all);
  for (int b = b0; b < b1; ++b) {
    const int n = sm_rank[b];
    sm_rank[b] = at;
    at += n;
  }
  long long total = all, before = 0;
  if (ctas > 1) {
    if (tid == 0) sm_total = all;
    cluster_sync();                         // every CTA has counted its pages
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
  for (int b = tid; b < B; b += SH_THREADS) a.lens_out[first + b] = sm_keep[b];
  if (rank == 0 && tid == 0) {
    const long long n = count + total;
    a.counts_out[0] = static_cast<int>(n < a.stack_size ? n : a.stack_size);
    a.counts_out[1] = static_cast<int>(n < a.stack_size ? 0 : n - a.stack_size);
  }
  const long long top = count + total - 1 - before;
  each([&](Ints b, Rows row) {
#pragma unroll
    for (int u = 0; u < SH_ROWS; ++u) {
      if (b[u] >= B) break;
      int i_th = sm_rank[b[u]];
#pragma unroll
      for (int i = 0; i < SH_BATCH; ++i) {
        const unsigned have = __ballot_sync(0xFFFFFFFFu, page[u][i] >= 0);
        if (page[u][i] >= 0) {
          const long long to = top - (i_th + __popc(have & ((1u << lane) - 1u)));
          if (to < a.stack_size) a.stack[to] = page[u][i];
          row[u][32 * i + lane] = -1;
        }
        i_th += __popc(have);
      }
      __syncwarp();
      if (lane == 0) sm_rank[b[u]] = i_th;  // (the row may go on)
      __syncwarp();
    }
  });
  __syncwarp();
  if (ctas > 1) cluster_wait();             // nobody reads this CTA's total any more
}

__global__ void __launch_bounds__(SH_THREADS) kv_fork_kernel(const ShareArgs a) {
  extern __shared__ int sm_claim[];         // per request: the fork that makes it, or none
  __shared__ int sm_served;
  constexpr int NONE = 0x7FFFFFFF;
  wait_for_stream();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, ctas = gridDim.x, share = share_of(a.requests, ctas);
  const int first = min(a.requests, rank * share), B = min(share, a.requests - first);
  int* sm_n = sm_claim + a.requests;        // per request of this CTA: its tokens as a fork
  if (tid == 0) sm_served = 0;
  for (int b = tid; b < a.requests; b += SH_THREADS) sm_claim[b] = NONE;
  __syncthreads();
  // every CTA goes over all forks: of several that name one request the first is it
  for (int i = tid; i < a.forks; i += SH_THREADS) {
    const int s = a.src[i], d = a.dst[i];
    const bool ok = s >= 0 && s < a.requests && d >= 0 && d < a.requests && s != d &&
                    a.lens[d] == 0 && a.lens[s] >= 0;
    if (ok) atomicMin(sm_claim + d, i);
  }
  __syncthreads();
  const long long capacity = a.width << a.page_shift;
  for (int b = tid; b < B; b += SH_THREADS) {
    const int i = sm_claim[first + b];
    int n = a.lens[first + b];
    if (i != NONE) {
      n = max(0, min(a.keep[i], a.lens[a.src[i]]));
      if (n > capacity) n = static_cast<int>(capacity);
    }
    sm_n[b] = n;
  }
  share_sync();                             // every CTA has read the lengths
  for (int b = tid; b < B; b += SH_THREADS) a.lens_out[first + b] = sm_n[b];
  if (rank == 0) {
    int served = 0;
    for (int b = tid; b < a.requests; b += SH_THREADS) served += sm_claim[b] != NONE;
    if (served) atomicAdd(&sm_served, served);
    __syncthreads();
    if (tid == 0) a.counts_out[0] = a.forks - sm_served;
  }
  for (int base = warp; base < B; base += SH_WARPS * SH_ROWS) {
    int n[SH_ROWS], most = 0;
    const int* from[SH_ROWS];
    int* to[SH_ROWS];
#pragma unroll
    for (int u = 0; u < SH_ROWS; ++u) {
      const int b = base + u * SH_WARPS;
      const int i = b < B ? sm_claim[first + b] : NONE;
      n[u] = 0;
      from[u] = to[u] = nullptr;
      if (i != NONE) {
        n[u] = static_cast<int>(share_blocks(sm_n[b], a.page_shift, a.width));
        from[u] = a.table + static_cast<long long>(a.src[i]) * a.table_stride;
        to[u] = a.table + static_cast<long long>(first + b) * a.table_stride;
      }
      most = max(most, n[u]);
    }
    for (int k0 = lane; k0 < most; k0 += SH_SPAN) {
      int page[SH_ROWS][SH_BATCH];
#pragma unroll
      for (int u = 0; u < SH_ROWS; ++u)
#pragma unroll
        for (int i = 0; i < SH_BATCH; ++i) page[u][i] = k0 + 32 * i < n[u] ? from[u][k0 + 32 * i] : -1;
#pragma unroll
      for (int u = 0; u < SH_ROWS; ++u)
#pragma unroll
        for (int i = 0; i < SH_BATCH; ++i) {
          if (k0 + 32 * i < n[u]) to[u][k0 + 32 * i] = page[u][i];
          if (page[u][i] >= 0 && page[u][i] < a.pages) atomicAdd(a.refs + page[u][i], 1);
        }
    }
  }
}

// One CTA: its steps are short and all depend on all requests.
__global__ void __launch_bounds__(SH_THREADS) kv_own_kernel(const ShareArgs a) {
  extern __shared__ int sm_page[];          // per request: the page it is about to write if others
                                            // hold it (-1: none), -2 - that for its keeper
  __shared__ int sm_scan[SH_WARPS];
  __shared__ int sm_cut, sm_served, sm_refused;
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the copies' CTAs may come and wait
  const int tid = threadIdx.x, B = a.requests, P = 1 << a.page_shift;
  const int per = (B + SH_THREADS - 1) / SH_THREADS;
  const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
  long long avail = *a.count;
  avail = avail < 0 ? 0 : (avail > a.stack_size ? a.stack_size : avail);
  if (tid == 0) {
    sm_cut = B;
    sm_served = sm_refused = 0;
  }
  auto entry = [&](int b, int len) {
    return a.table + static_cast<long long>(b) * a.table_stride + (len >> a.page_shift);
  };
  for (int b = tid; b < B; b += SH_THREADS) {
    const int len = a.lens[b];
    int page = -1;
    if (a.change[b] > 0 && len > 0 && (len & (P - 1)) && (len >> a.page_shift) < a.width) {
      page = *entry(b, len);
      if (page < 0 || page >= a.pages || a.refs[page] <= 0) page = -1;
    }
    sm_page[b] = page;
  }
  __syncthreads();
  for (int b = tid; b < B; b += SH_THREADS)
    if (sm_page[b] >= 0) atomicSub(a.refs + sm_page[b], 1);
  __syncthreads();
  for (int b = tid; b < B; b += SH_THREADS)
    if (sm_page[b] >= 0 && __ldcg(a.refs + sm_page[b]) < 0) atomicMin(a.refs + sm_page[b], -2 - b);
  __syncthreads();
  for (int b = tid; b < B; b += SH_THREADS)
    if (sm_page[b] >= 0 && __ldcg(a.refs + sm_page[b]) == -2 - b) sm_page[b] = -2 - sm_page[b];
  __syncthreads();
  int mine = 0, all;
  for (int b = b0; b < b1; ++b) {
    mine += sm_page[b] >= 0;
    if (sm_page[b] < -1) atomicExch(a.refs + (-2 - sm_page[b]), 0);
  }
  const int at = share_scan(mine, sm_scan, all);
  // the first that finds no page: it and all behind it that would write a page that others
  // hold are refused
  {
    long long i = at;
    for (int b = b0; b < b1; ++b) {
      if (sm_page[b] < 0) continue;
      if (i >= avail) {
        atomicMin(&sm_cut, b);
        break;
      }
      ++i;
    }
  }
  __syncthreads();
  const int cut = sm_cut;
  int i_th = at, served = 0, refused = 0;
  for (int b = b0; b < b1; ++b) {
    const int held = sm_page[b];
    int from = -1, to = -1, tokens = -1;
    bool no = false;
    if (held != -1) {
      no = b >= cut;
      refused += no;
      if (held >= 0) {
        if (no) {
          atomicAdd(a.refs + held, 1);      // it goes on holding the page
        } else {
          const int len = a.lens[b];
          from = held;
          to = a.stack[avail - 1 - i_th];
          tokens = len & (P - 1);
          *entry(b, len) = to;
          ++i_th;
          ++served;
        }
      }
    }
    a.lens_out[b] = no ? 0 : a.change[b];
    a.copies[3 * b] = from;
    a.copies[3 * b + 1] = to;
    a.copies[3 * b + 2] = tokens;
  }
  if (served) atomicAdd(&sm_served, served);
  if (refused) atomicAdd(&sm_refused, refused);
  __syncthreads();
  if (tid == 0) {
    a.counts_out[0] = static_cast<int>(avail) - sm_served;
    a.counts_out[1] = sm_refused;
  }
}

// The copies of own's plan: the first tokens of a page, for `heads` heads a CTA, of K
// or of V (blockIdx.z).  A head's tokens are contiguous.
constexpr int CP_THREADS = 256, CP_BATCH = 4;
__global__ void __launch_bounds__(CP_THREADS)
kv_copy_kernel(const KvCache c, const int* copies, int heads_per_cta, int page_shift, int d_shift) {
  wait_for_stream();
  const int* job = copies + 3ll * blockIdx.x;
  const int from = __ldcg(job), to = __ldcg(job + 1), tokens = __ldcg(job + 2);
  if (from < 0 || to < 0 || from >= c.pages || to >= c.pages) return;
  const int h0 = blockIdx.y * heads_per_cta;
  const int heads = min(heads_per_cta, static_cast<int>(c.heads) - h0);
  uint8_t* codes = blockIdx.z ? c.v : c.k;
  uint8_t* scales = blockIdx.z ? c.v_scales : c.k_scales;
  const long long a = from * c.heads + h0, b = to * c.heads + h0;
  for (int h = threadIdx.x; h < heads; h += CP_THREADS) scales[b + h] = scales[a + h];
  const int unit_shift = page_shift + d_shift - 4, row = tokens << (d_shift - 4);   // 16-byte chunks
  const uint4* src = reinterpret_cast<const uint4*>(codes) + (a << unit_shift);
  uint4* dst = reinterpret_cast<uint4*>(codes) + (b << unit_shift);
  const int n = heads * row;
  for (int i0 = threadIdx.x; i0 < n; i0 += CP_THREADS * CP_BATCH) {
    uint4 v[CP_BATCH];
    long long at[CP_BATCH];
#pragma unroll
    for (int u = 0; u < CP_BATCH; ++u) {
      const int i = i0 + u * CP_THREADS;
      if (i >= n) break;
      const int h = i / row;
      at[u] = (static_cast<long long>(h) << unit_shift) + (i - h * row);
      v[u] = src[at[u]];
    }
#pragma unroll
    for (int u = 0; u < CP_BATCH; ++u)
      if (i0 + u * CP_THREADS < n) dst[at[u]] = v[u];
  }
}

// Each kernel's limit of shared memory belongs to the kernel, not to the launch: it is
// set once, to the most that any call needs.
cudaError_t launch_share(void (*kern)(const ShareArgs), const ShareArgs& a, int ctas, size_t smem,
                         size_t most_smem, std::atomic<bool> (&set)[64], cudaStream_t st) {
  if (smem > SH_SMEM_FREE) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !set[dev].load(std::memory_order_relaxed)) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(most_smem));
      if (e != cudaSuccess) return e;
      if (dev < 64) set[dev].store(true, std::memory_order_relaxed);
    }
  }
  return launch_early(kern, dim3(static_cast<unsigned>(ctas)), SH_THREADS, smem, ctas, st, a);
}

// One CTA where its warps look after all requests at once: a cluster's barriers
// take longer than sharing out saves.  16 where that is fewer rows for each warp and the
// device has room for such a cluster (more than the 8 that every device of this
// architecture holds): eight samples of each of 18, 25, 36, 64, 128 and 256 prompts take
// 22.9, 24.3, 27.1, 35.7, 50.6 and 84.3 us, with 8 CTAs 22.4, 24.4, 27.8, 38.2, 60.4 and 99.7.
int share_ctas(void (*kern)(const ShareArgs), int64_t requests, std::atomic<int> (&most)[64]) {
  if (requests <= SH_WARPS * SH_ROWS) return 1;
  int dev = 0;
  if (requests <= SH_CLUSTER * SH_WARPS || cudaGetDevice(&dev) != cudaSuccess || dev >= 64)
    return SH_CLUSTER;
  int ctas = most[dev].load(std::memory_order_relaxed);
  if (ctas == 0) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = SH_WIDE;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SH_WIDE);
    cfg.blockDim = dim3(SH_THREADS);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    const bool wide =
        cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0;
    if (!wide) cudaGetLastError();
    ctas = wide ? SH_WIDE : SH_CLUSTER;
    most[dev].store(ctas, std::memory_order_relaxed);
  }
  return ctas;
}

}  // namespace

cudaError_t launch_kv_release(const KvShare& q, cudaStream_t st) {
  ShareArgs a{};
  a.lens = q.lens;
  a.change = q.change;
  a.table = q.table;
  a.table_stride = q.table_stride;
  a.width = q.width;
  a.stack = q.stack;
  a.stack_size = q.stack_size;
  a.count = q.count;
  a.refs = q.refs;
  a.pages = static_cast<int>(q.pages);
  a.page_shift = kv_page_shift(q.page);
  a.requests = static_cast<int>(q.requests);
  a.lens_out = q.lens_out;
  a.counts_out = q.counts_out;
  static std::atomic<bool> set[64] = {};
  static std::atomic<int> most[64] = {};
  const int ctas = share_ctas(kv_release_kernel, q.requests, most);
  static_assert(3 * SH_MAX_REQUESTS / SH_CLUSTER * sizeof(int) <= SH_SMEM_FREE, "");
  return launch_share(kv_release_kernel, a, ctas, 3 * share_of(a.requests, ctas) * sizeof(int), 0, set, st);
}

cudaError_t launch_kv_fork(const KvShare& q, cudaStream_t st) {
  ShareArgs a{};
  a.lens = q.lens;
  a.src = q.src;
  a.dst = q.dst;
  a.keep = q.change;
  a.forks = static_cast<int>(q.forks);
  a.table = q.table;
  a.table_stride = q.table_stride;
  a.width = q.width;
  a.refs = q.refs;
  a.pages = static_cast<int>(q.pages);
  a.page_shift = kv_page_shift(q.page);
  a.requests = static_cast<int>(q.requests);
  a.lens_out = q.lens_out;
  a.counts_out = q.counts_out;
  static std::atomic<bool> set[64] = {};
  static std::atomic<int> most[64] = {};
  const int ctas = share_ctas(kv_fork_kernel, q.requests, most);
  return launch_share(kv_fork_kernel, a, ctas, (a.requests + share_of(a.requests, ctas)) * sizeof(int),
                      (SH_MAX_REQUESTS + SH_MAX_REQUESTS / SH_CLUSTER) * sizeof(int), set, st);
}

cudaError_t launch_kv_own(const KvCache& c, const KvShare& q, cudaStream_t st) {
  ShareArgs a{};
  a.lens = q.lens;
  a.change = q.change;
  a.table = q.table;
  a.table_stride = q.table_stride;
  a.width = q.width;
  a.stack = q.stack;
  a.stack_size = q.stack_size;
  a.count = q.count;
  a.refs = q.refs;
  a.pages = static_cast<int>(c.pages);
  a.page_shift = kv_page_shift(c.page);
  a.requests = static_cast<int>(q.requests);
  a.lens_out = q.lens_out;
  a.copies = q.copies;
  a.counts_out = q.counts_out;
  static std::atomic<bool> set[64] = {};
  cudaError_t e = launch_share(kv_own_kernel, a, 1, a.requests * sizeof(int),
                               SH_MAX_REQUESTS * sizeof(int), set, st);
  if (e != cudaSuccess || a.requests == 0) return e;
  // a head or more a CTA: as many as leave about four CTAs for each of the 152 SMs
  // if every request were to copy
  int64_t per = 1;
  while (per < c.heads && a.requests * 2 * (c.heads / per) > 1216) per *= 2;
  const dim3 grid(static_cast<unsigned>(a.requests), static_cast<unsigned>((c.heads + per - 1) / per), 2);
  return launch_early(kv_copy_kernel, grid, CP_THREADS, 0, 1, st, c, static_cast<const int*>(q.copies),
                      static_cast<int>(per), a.page_shift, c.d == 64 ? 6 : 7);
}

}  // namespace mxk
