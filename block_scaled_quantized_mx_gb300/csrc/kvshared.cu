// kvshared.cu -- attention over the paged cache for groups of requests that share a
// prefix: the prefix's keys are read once for all of a group's rows.
//
// With the keys of a row in two sets, P (the prefix) and S (its own),
//   o = (w_P O_P + w_S O_S) / (w_P l_P + w_S l_S),  w_i = 2^(m_i - max(m_P, m_S)),
// O_i = sum_j 2^(x_j - m_i) v_j and l_i = sum_j 2^(x_j - m_i) over the set's keys: the
// identity behind the running softmax.  So three steps, each the next one's
// programmatic dependency:
//   plan     how much of each prefix its group's rows of the table agree on and all of its
//            rows may see, and those rows (consecutive requests' are consecutive) -- a few
//            integers;
//   prefix   the kernels of kvattn.cu or kvprompt.cu with a group in a request's place:
//            all of its rows, over the prefix; (O, m, l) per row are left in memory;
//   own      the same kernels over each request's keys behind the prefix; who writes a
//            row takes the prefix's (O, m, l) up.
// Precision: as those kernels have it; (O, m, l) and their joining are fp32.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "kv_common.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int SP_THREADS = 1024;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_MAX = 16384;               // requests, and groups
constexpr int SP_CLUSTER = 8;               // CTAs to a group, where there are few
constexpr int SP_MANY_GROUPS = 64;
constexpr int SP_BATCH = 8;                 // table entries of a lane on their way together

struct PlanArgs {
  const int* lens;
  const int* cu;
  const int* groups;
  const int* shared;
  const int* table;
  long long table_stride;
  int requests;
  int capacity;               // tokens a table row holds
  int page_shift;
  int* start;                 // per request: keys of its group's prefix, 0 where it has none
  int* rows;                  // per group: its rows' first and end
  int* plens;                 // per group: its prefix's keys
  int* row_of;                // per group: the request in whose row of the table the prefix is found
};

__device__ __forceinline__ int plan_reduce(int v, int* sm, bool least) {
  v = least ? __reduce_min_sync(0xFFFFFFFFu, v) : __reduce_max_sync(0xFFFFFFFFu, v);
  __syncthreads();                          // sm is free
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[threadIdx.x & 31];
  static_assert(SP_WARPS == 32, "a lane for each warp");
  return least ? __reduce_min_sync(0xFFFFFFFFu, v) : __reduce_max_sync(0xFFFFFFFFu, v);
}

// One group to a CTA or to a cluster.  Its requests are groups[g] .. groups[g + 1] - 1,
// offsets taken in order: one below an earlier one counts as that one.  Its prefix is what
// `shared` says, what stands in front of all its rows, and what the rows of the table agree on,
// whichever is least: a wrong word about a prefix costs time, not the answer.
__global__ void __launch_bounds__(SP_THREADS) kv_plan_kernel(const PlanArgs a) {
  __shared__ int sm[SP_WARPS];
  __shared__ int sm_agree;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, B = a.requests;
  const int rank = blockIdx.x, ctas = gridDim.x, g = blockIdx.y;
  int top = 0;
  for (int i = tid; i <= g; i += SP_THREADS) top = max(top, max(0, min(a.groups[i], B)));
  const int r0 = plan_reduce(top, sm, false);
  const int r1 = max(r0, max(0, min(a.groups[g + 1], B)));
  // the tokens that stand in front of every row of the group
  int most = 0x7FFFFFFF, with_rows = 0;
  for (int b = r0 + tid; b < r1; b += SP_THREADS) {
    const int n = a.cu[b + 1] - a.cu[b];
    if (n > 0) {
      most = min(most, max(0, min(a.lens[b], a.capacity)) - n);
      ++with_rows;
    }
  }
  most = min(plan_reduce(most, sm, true), a.shared[g]);
  if (plan_reduce(with_rows, sm, false) < 2 && __syncthreads_count(with_rows) < 2) most = 0;
  // the first entry on which a row of the table differs from the group's first
  const int pages = most <= 0 ? 0 : static_cast<int>((most + (1ll << a.page_shift) - 1) >> a.page_shift);
  const int* first = a.table + r0 * a.table_stride;
  const int chunks = (pages + 32 * SP_BATCH - 1) / (32 * SP_BATCH);
  int agree = pages;
  for (long long i = rank * SP_WARPS + (tid >> 5); i < static_cast<long long>(chunks) * (r1 - r0 - 1);
       i += ctas * SP_WARPS) {
    const int b = r0 + 1 + static_cast<int>(i / chunks);
    const int j0 = static_cast<int>(i % chunks) * 32 * SP_BATCH + lane;
    const int* row = a.table + b * a.table_stride;
    int own[SP_BATCH], ref[SP_BATCH];
#pragma unroll
    for (int u = 0; u < SP_BATCH; ++u) {
      own[u] = ref[u] = 0;
      if (j0 + 32 * u < pages) {
        own[u] = row[j0 + 32 * u];
        ref[u] = first[j0 + 32 * u];
      }
    }
#pragma unroll
    for (int u = SP_BATCH - 1; u >= 0; --u)
      if (own[u] != ref[u]) agree = min(agree, j0 + 32 * u);
  }
  agree = plan_reduce(agree, sm, true);
  if (ctas > 1) {
    if (tid == 0) sm_agree = agree;
    cluster_sync();
    agree = lane < ctas ? ld_shared_cluster_s32(map_to_cta(smem_u32(&sm_agree), lane)) : pages;
    agree = __reduce_min_sync(0xFFFFFFFFu, agree);
    cluster_arrive();
  }
  const int keys = agree < pages ? agree << a.page_shift : max(0, most);
  if (rank == 0) {
    if (tid == 0) {
      const int q0 = a.cu[r0];
      a.rows[2 * g] = q0;
      a.rows[2 * g + 1] = keys > 0 ? a.cu[r1] : q0;
      a.plens[g] = keys;
      a.row_of[g] = r0;
    }
    for (int b = r0 + tid; b < r1; b += SP_THREADS) a.start[b] = keys;
    // requests of no group
    if (g == 0)
      for (int b = tid; b < r0; b += SP_THREADS) a.start[b] = 0;
    if (g == gridDim.y - 1)
      for (int b = r1 + tid; b < B; b += SP_THREADS) a.start[b] = 0;
  }
  __syncwarp();
  if (ctas > 1) cluster_wait();             // nobody reads this CTA's word any more
}

int64_t up32(int64_t n) { return (n + 31) / 32 * 32; }

// The workspace: the plan's integers, the rows' states, the two passes' scratch.
struct Layout {
  int64_t start, rows, plens, row_of, o, ml, prefix, own, total;
};
// rows of a group at the most: with one group all tokens
Layout layout_of(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_q,
                 int64_t requests, int64_t groups) {
  Layout l;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up32(bytes);
    return here;
  };
  l.start = take(4 * requests);
  l.rows = take(8 * groups);
  l.plens = take(4 * groups);
  l.row_of = take(4 * groups);
  l.o = take(4 * tokens * q_heads * d);
  l.ml = take(8 * tokens * q_heads);
  l.prefix = take(static_cast<int64_t>(kv_pass_workspace_bytes(q_heads / kv_heads, d, tokens)));
  l.own = take(static_cast<int64_t>(kv_pass_workspace_bytes(q_heads / kv_heads, d, max_q)));
  l.total = at;
  return l;
}

}  // namespace

size_t kv_attention_shared_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d,
                                           int64_t max_q, int64_t requests, int64_t groups) {
  if (requests > SP_MAX || groups > SP_MAX) return 0;
  // (16 bytes to bring a workspace that begins at a 16-byte boundary to a 32-byte one)
  return static_cast<size_t>(layout_of(tokens, q_heads, kv_heads, d, max_q, requests, groups).total + 16);
}

cudaError_t launch_kv_attention_shared(const KvAttn& q, const KvGroups& g, cudaStream_t st) {
  const int64_t kv_heads = q.cache.heads;
  const size_t need = kv_attention_shared_workspace_bytes(q.tokens, q.q_heads, kv_heads, q.cache.d, q.max_q,
                                                          q.requests, g.n);
  // without groups or room for the states: each request for itself
  if (g.n == 0 || need == 0 || q.ws == nullptr || q.ws_bytes < need) return launch_kv_attention(q, st);
  const Layout l = layout_of(q.tokens, q.q_heads, kv_heads, q.cache.d, q.max_q, q.requests, g.n);
  char* ws = static_cast<char*>(q.ws) + (reinterpret_cast<uintptr_t>(q.ws) & 16);
  PlanArgs p{};
  p.lens = q.lens;
  p.cu = q.cu;
  p.groups = g.groups;
  p.shared = g.shared;
  p.table = q.table;
  p.table_stride = q.table_stride;
  p.page_shift = kv_page_shift(q.cache.page);
  p.requests = static_cast<int>(q.requests);
  const int64_t most = q.width << kv_page_shift(q.cache.page);
  p.capacity = static_cast<int>(most < 0x7FFFFF00 ? most : 0x7FFFFF00);
  p.start = reinterpret_cast<int*>(ws + l.start);
  p.rows = reinterpret_cast<int*>(ws + l.rows);
  p.plens = reinterpret_cast<int*>(ws + l.plens);
  p.row_of = reinterpret_cast<int*>(ws + l.row_of);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(g.n > SP_MANY_GROUPS ? 1 : SP_CLUSTER, static_cast<unsigned>(g.n));
  cfg.blockDim = dim3(SP_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cfg.gridDim.x;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv_plan_kernel, p);
  if (e != cudaSuccess) return e;
  KvPassArgs pass{};
  pass.state.o = reinterpret_cast<float*>(ws + l.o);
  pass.state.ml = reinterpret_cast<float2*>(ws + l.ml);
  // prefixes: a group in a request's place, whose rows all see all of its keys
  KvAttn a = q;
  a.cu = p.rows;
  a.lens = p.plens;
  a.requests = g.n;
  a.max_q = std::max<int64_t>(1, q.tokens / g.n);
  a.causal = 0;
  a.o_ts = a.o_hs = 0;                      // O is not written
  a.ws = ws + l.prefix;
  a.ws_bytes = static_cast<size_t>(l.own - l.prefix);
  pass.row_of = p.row_of;
  pass.cu_step = 2;
  pass.state.pass = KV_PREFIX;
  e = launch_kv_pass(a, pass, st);
  if (e != cudaSuccess) return e;
  a = q;
  a.ws = ws + l.own;
  a.ws_bytes = static_cast<size_t>(l.total - l.own);
  pass.start = p.start;
  pass.row_of = nullptr;
  pass.cu_step = 1;
  pass.state.pass = KV_OWN;
  return launch_kv_pass(a, pass, st);
}

}  // namespace mxk
