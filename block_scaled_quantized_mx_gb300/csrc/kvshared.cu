// kvshared.cu -- attention over the paged cache for groups of requests that share a
// prefix: the prefix's keys are read once for all of a group's rows.
//
// With the keys of a row in two sets, P (the prefix) and S (its own),
//   o = (w_P O_P + w_S O_S) / (w_P l_P + w_S l_S),  w_i = 2^(m_i - max(m_P, m_S)),
// O_i = sum_j 2^(x_j - m_i) v_j and l_i = sum_j 2^(x_j - m_i) over the set's keys: the
// identity behind the running softmax, and the same for the parts of a set.  Three or four
// steps, each the next one's programmatic dependency:
//   plan   how much of each prefix its group's rows of the table agree on and all of its
//          rows may see, and a list for the kernels of kvattn.cu and kvprompt.cu: an
//          entry for each group (all of its rows, which are consecutive, over the prefix)
//          and one for each request (its rows over its keys behind the prefix);
//   pass   one of those kernels over the list, or one over each half of it, where the rows
//          of groups and of requests want different ones.  Rows without a prefix are
//          written, unless their unit is cut; the others leave (O, m, l) in memory, in
//          as many parts as CTAs shared their units;
//   join   each such row from the parts of both sets.
// Precision: as those kernels have it; (O, m, l) and their joining are fp32, in a fixed
// order.
// Bound: HBM for the own keys, the tensor rate or HBM for the prefix; between them the four
// launches.  Measured with 32 heads on 8 cache heads of 128, E4M3 (mx_kv_attention,
// for which a prefix that fits in L2 comes from there): 64 requests behind 8192 tokens with up to 512
// of their own 43 us (113), of which the plan takes 3.5, both passes, side by side, 27, the
// join 6.5; 128 requests with four drafts behind 32768 tokens, E5M2, 283 us (1300), 266 of them the
// prompt kernel on 128 SMs, at 0.62 of their bf16 rate; 16 groups of eight behind up
// to 3000 tokens, 16 heads of 64, int8, pages of 16, 44 us (120).
// (With a join for each pass, the own pass taking the prefix's states up as it wrote: 58, 315,
// 82; with the prefix's pass on all SMs and the own one behind it: 50; with the own one
// on the SMs that are left by six entries a CTA: 48, 297.)
#include <algorithm>
#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "kv_common.cuh"
#include "kv_kernel.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int SP_THREADS = 1024;
constexpr int SP_WARPS = SP_THREADS / 32;
constexpr int SP_MAX = 16384;               // requests, and groups
// CTAs to a group where its rows of the table are long, and the groups few
constexpr int SP_CLUSTER = 8;
constexpr int SP_MANY_GROUPS = 64;
constexpr int64_t SP_ENTRIES = 16384;       // of the table, for one CTA
constexpr int SP_BATCH = 8;                 // table entries of a lane on their way together

// A prefix is worth a pass where it saves this many bytes of reads.  They come from L2
// for all requests but one, so that mx_kv_attention loses little by short ones.  Measured
// with 8 cache heads of 128 values, one group (shared against mx_kv_attention; MiB saved):
// 4 requests, 8192 keys 19.5 against 16.6 us (48); 16, 2048 keys 25.5 against 17.1 (60), 4096
// 27.1 against 23.4 (120), 8192 30 against 36 (240); 64, 512 keys 28 against 20 (63), 1024 29 against
// 27 (126), 2048 35 against 42 (252), 8192 43 against 113 (1008); 64 values 29 against 35 (184).
constexpr int64_t SP_WORTH = 150 << 20;
std::atomic<int64_t> g_worth{SP_WORTH};
// Nor is it where the requests' rows fill the prompt kernel's units of 256 by themselves: its time
// is then that of the products, which sharing does not save.  Rows of each request, on the average;
// measured (32 requests behind 4096 tokens; shared against mx_kv_attention): 36 rows 55 against
// 109 us, 64 70 against 111, 128 106 against 114, 256 185 against 146; behind 8192, one cache
// head to eight, 128 rows 164 against 202; 64 behind 8192, 256 rows 544 against 469.
constexpr int64_t SP_MOST_ROWS = 192;

// SM-microseconds of an entry of either pass, for sharing the SMs out between them (a unit's
// blocks of 128 keys and four more; its tiles and two more).  Fitted where one or the other
// bounded the whole, with 8 cache heads, 16 to 256 requests of up to 2048 tokens, 52 to 140 SMs
// for prefixes of 2048 to 32768: 1.8 to 2.0, with 64 values 1.54 to 1.63; 0.35 to 0.41 and 0.8 to
// 0.95 with 8 and 16 rows a unit, with 64 values about 0.7 of that; int8 codes 1.0 to 1.2.  (With the requests' pass on
// the SMs that six entries a CTA left, 64 requests behind 8192 tokens took 48 us instead of 43,
// up to 2048 of their own behind 16384 77 instead of 62, 128 x 4 drafts behind 32768 297
// instead of 283.)
constexpr float SP_PREFIX_128 = 1.9f, SP_PREFIX_64 = 1.6f;
constexpr float SP_OWN_8 = 0.4f, SP_OWN_16 = 0.9f, SP_OWN_INT8 = 1.1f, SP_OWN_64 = 0.7f;

struct PlanArgs {
  const int* lens;
  const int* cu;
  const int* groups;
  const int* shared;
  const int* table;
  long long table_stride;
  int requests;
  int n;                      // groups
  int capacity;               // tokens a table row holds
  int page_shift;
  long long worth;            // keys times requests that are spared them, of all groups, to be shared at all
  KvEntry* list;              // n for the groups, then the requests'
  // what the passes are expected to take, where they run beside one another (split)
  int split;
  int heads, group;           // of the cache, query heads of each
  int own_rows;               // of a unit of the requests' pass
  float own_entry, prefix_entry;   // SM-microseconds of a tile, of a block of 256 rows
};

// The least a and c and the sum of b over the block's threads.  `sm`: of this call alone.
__device__ __forceinline__ void plan_reduce(int& a, int& b, int& c, int4* sm) {
  const int la = __reduce_min_sync(0xFFFFFFFFu, a), sb = __reduce_add_sync(0xFFFFFFFFu, b);
  const int lc = __reduce_min_sync(0xFFFFFFFFu, c);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = make_int4(la, sb, lc, 0);
  __syncthreads();
  const int4 v = sm[threadIdx.x & 31];
  static_assert(SP_WARPS == 32, "a lane for each warp");
  a = __reduce_min_sync(0xFFFFFFFFu, v.x);
  b = __reduce_add_sync(0xFFFFFFFFu, v.y);
  c = __reduce_min_sync(0xFFFFFFFFu, v.z);
}

// The sum over the block's threads, in a fixed order.
__device__ __forceinline__ float plan_sum(float v, float* sm) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = sm[threadIdx.x & 31];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// The prompt kernel's units of so many rows.  Their 256 rows go in halves: one alone takes
// 0.74 of the time of both.
__device__ __forceinline__ float plan_units_256(float rows) {
  const float full = floorf(rows / 256.0f), rest = rows - 256.0f * full;
  return full + (rest > 128.0f ? 1.0f : rest > 0.0f ? 0.74f : 0.0f);
}

// One group to a CTA or to a cluster.  Its requests are groups[g] .. groups[g + 1] - 1,
// offsets taken in order: one below an earlier one counts as that one.  Its prefix is what
// `shared` says, what stands in front of all its rows, and what the rows of the table of its
// requests that have rows agree on, whichever is least (a wrong word about a prefix costs
// time, not the answer); or nothing, if that is too little for a pass.  A request without
// rows, which may have ended and hold nothing, has no say.
__global__ void __launch_bounds__(SP_THREADS) kv_plan_kernel(const PlanArgs a) {
  __shared__ int4 sm[3][SP_WARPS];
  __shared__ int sm_agree;
  __shared__ float sm_own[SP_WARPS];
  wait_for_stream();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, lane = tid & 31, B = a.requests;
  const int rank = blockIdx.x, ctas = gridDim.x, g = blockIdx.y;
  int r0 = 0, several = 0, none = 0;         // several: groups of two requests or more
#pragma unroll 1                              // (unrolled, its code took 0.3 us to fetch)
  for (int i = tid; i < a.n; i += SP_THREADS) {
    const int from = max(0, min(a.groups[i], B)), to = max(0, min(a.groups[i + 1], B));
    if (i <= g) r0 = min(r0, -from);
    several += to - from >= 2;
  }
  const int edge = max(0, min(a.groups[g + 1], B)), said = a.shared[g];
  // (with the offsets, before it is known which requests matter: the tokens in front of
  // a request's rows)
  auto in_front = [&](int b) {
    const int n = a.cu[b + 1] - a.cu[b];
    return n > 0 ? max(0, min(a.lens[b], a.capacity)) - n : 0x7FFFFFFF;
  };
  const int mine = tid < B ? in_front(tid) : 0x7FFFFFFF;
  plan_reduce(r0, several, none, sm[0]);
  r0 = -r0;
  const int r1 = max(r0, edge);
  // the tokens that stand in front of every row of the group, and its first request with rows
  int most = 0x7FFFFFFF, with_rows = 0, lead = 0x7FFFFFFF;
  auto count = [&](int b, int tokens) {
    if (tokens == 0x7FFFFFFF) return;
    most = min(most, tokens);
    lead = min(lead, b);
    ++with_rows;
  };
  if (tid >= r0 && tid < r1) count(tid, mine);
  for (int b = tid + SP_THREADS; b < r1; b += SP_THREADS)
    if (b >= r0) count(b, in_front(b));
  plan_reduce(most, with_rows, lead, sm[1]);
  most = with_rows < 2 ? 0 : min(most, said);
  // the first entry on which a row of the table differs from that request's
  const int pages = most <= 0 ? 0 : static_cast<int>((most + (1ll << a.page_shift) - 1) >> a.page_shift);
  const int* first = a.table + (pages > 0 ? lead : 0) * a.table_stride;
  const int chunks = (pages + 32 * SP_BATCH - 1) / (32 * SP_BATCH);
  int agree = pages;
  for (long long i = rank * SP_WARPS + (tid >> 5); i < static_cast<long long>(chunks) * (r1 - 1 - lead);
       i += ctas * SP_WARPS) {
    const int b = lead + 1 + static_cast<int>(i / chunks);
    const int j0 = static_cast<int>(i % chunks) * 32 * SP_BATCH + lane;
    const int* row = a.table + b * a.table_stride;
    const bool has_rows = a.cu[b + 1] > a.cu[b];   // (read with the entries)
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
      if (has_rows && own[u] != ref[u]) agree = min(agree, j0 + 32 * u);
  }
  plan_reduce(agree, none, none, sm[2]);
  if (ctas > 1) {
    if (tid == 0) sm_agree = agree;
    cluster_sync();
    agree = lane < ctas ? ld_shared_cluster_s32(map_to_cta(smem_u32(&sm_agree), lane)) : pages;
    agree = __reduce_min_sync(0xFFFFFFFFu, agree);
    cluster_arrive();
  }
  int keys = agree < pages ? agree << a.page_shift : max(0, most);
  // (what is asked of all, as if the groups that can share anything were alike)
  if (static_cast<long long>(keys) * (with_rows - 1) * max(1, several) < a.worth) keys = 0;
  auto entry = [&](int i, int q0, int q1, int len, int start, int row, int prefix, float t0, float t1) {
    int4* e = reinterpret_cast<int4*>(a.list + i);
    e[0] = make_int4(q0, q1, len, start);
    e[1] = make_int4(row, prefix, __float_as_int(t0), __float_as_int(t1));
  };
  float own = 0.0f;                         // entries of the requests' pass
  auto request = [&](int b, int start) {
    const int q0 = a.cu[b], q1 = a.cu[b + 1], len = a.lens[b];
    entry(a.n + b, q0, q1, len, start, b, 0, 0.0f, 0.0f);
    if (a.split && q1 > q0) {
      const int from = start >> a.page_shift << a.page_shift;
      const int tiles = max(1, (max(0, min(len, a.capacity) - from) + 127) / 128);
      const float rows = static_cast<float>(q1 - q0) * a.group;
      own += a.own_rows == 256 ? plan_units_256(rows) * (4 + tiles) : ceilf(rows / a.own_rows) * (2 + tiles);
    }
  };
  if (rank == 0) {
    for (int b = r0 + tid; b < r1; b += SP_THREADS) request(b, keys);
    // requests of no group
    if (g == 0)
      for (int b = tid; b < r0; b += SP_THREADS) request(b, 0);
    if (g == a.n - 1)
      for (int b = r1 + tid; b < B; b += SP_THREADS) request(b, 0);
    float prefix = 0.0f;
    if (a.split) {
      own = plan_sum(own, sm_own);
      prefix = plan_units_256(static_cast<float>(a.cu[r1] - a.cu[r0]) * a.group) * (4 + (keys + 127) / 128);
    }
    if (tid == 0)
      entry(g, a.cu[r0], keys > 0 ? a.cu[r1] : a.cu[r0], keys, 0, keys > 0 ? lead : r0, 1,
            keys > 0 ? prefix * a.heads * a.prefix_entry : 0.0f, own * a.heads * a.own_entry);
  }
  __syncwarp();
  if (ctas > 1) cluster_wait();             // nobody reads this CTA's word any more
}

// The parts of one set: where a pass's kernel (rows of a unit, CTAs) left them.
struct JoinSet {
  KvStates states;
  const float* parts;
  int unit;
  int ctas;
};
struct JoinArgs {
  JoinSet prefix, own;
  const int* cu;
  int requests;
  long long rows;             // tokens x q_heads
  int q_heads;
  void* O;
  int o_dtype;
  long long o_ts, o_hs;
};

constexpr int SJ_THREADS = 256, SJ_BATCH = 3;
constexpr int64_t SJ_FEW_ROWS = 4096;

// SJ_LANES lanes take eight columns of a row, each every SJ_LANES-th of its parts --
// the prefix's, then its own -- SJ_BATCH of them with their loads together, and meet by
// shuffles.  Four lanes where the rows are few: their parts then are many (64 rows of 32
// heads behind 8192 keys have 12 a row), and the wait for one read after the other bounds it; one
// lane where the rows fill the SMs (16384 rows of 5 parts: 25 us with four).
template <int D, int SJ_LANES>
__global__ void __launch_bounds__(SJ_THREADS) kv_join_states_kernel(const JoinArgs a) {
  wait_for_stream();
  const int tid = threadIdx.x, k = tid & (SJ_LANES - 1);
  const long long at = (static_cast<long long>(blockIdx.x) * SJ_THREADS + tid) / SJ_LANES;
  const long long row = at / (D / 8);
  const int col = 8 * static_cast<int>(at % (D / 8));
  if (row >= a.rows) return;                // (SJ_LANES lanes alike)
  const long long token = row / a.q_heads;
  const int head = static_cast<int>(row - token * a.q_heads);
  // (all of these at once: each is a read from L2)
  const int4 own = __ldcg(a.own.states.rec + row);
  int4 pre = __ldcg(a.prefix.states.rec + row);
  const int first = a.cu[0], end = a.cu[a.requests];
  if (token < first || token >= end) return;   // of no request: left as it is
  if (own.w & KV_REC_DONE) return;
  const bool has_prefix = (own.w & KV_REC_PREFIX) != 0;
  if (!has_prefix) pre = make_int4(0, 0, 0, 0);
  // (offsets that go up and down may leave a row without a word of this call's)
  auto sound = [](const int4& r, const JoinSet& s) {
    return r.z == 0 || (r.z > 1 && r.y >= 0 && r.y + r.z <= s.ctas && r.x >= 0 && r.x < 2 * s.ctas &&
                        (r.w & 0xFFFF) < s.unit);
  };
  if (!sound(own, a.own) || !sound(pre, a.prefix)) return;
  const int n_pre = has_prefix ? max(1, pre.z) : 0, n = n_pre + max(1, own.z);
  auto read = [&](int i, float& m, float& l, float (&v)[8]) {
    const bool of_prefix = i < n_pre;
    const JoinSet& s = of_prefix ? a.prefix : a.own;
    const int4 r = of_prefix ? pre : own;
    const int p = of_prefix ? i : i - n_pre, rr = r.w & 0xFFFF;
    if (r.z == 0) {
      const float2 ml = __ldcg(s.states.ml + row);
      m = ml.x;
      l = ml.y;
      ld_global_cg_v8(s.states.o + row * D + col, v);
    } else {
      const int slot = p == 0 ? r.x : 2 * (r.y + p);
      const float* part = s.parts + static_cast<long long>(slot) * s.unit * (D + 2);
      m = __ldcg(part + s.unit * D + rr);
      l = __ldcg(part + s.unit * (D + 1) + rr);
      // the prompt kernel's parts are [8 columns][row][column]
      const float* o = s.unit == 256 ? part + (col / 8 * 256 + rr) * 8 : part + rr * D + col;
      if ((reinterpret_cast<uintptr_t>(o) & 31) == 0) {
        ld_global_cg_v8(o, v);
      } else {
        const float4 x = ld_global_cg_f4(o), y = ld_global_cg_f4(o + 4);
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
        v[4] = y.x;
        v[5] = y.y;
        v[6] = y.z;
        v[7] = y.w;
      }
    }
  };
  float top = -INFINITY, sum = 0.0f, acc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0.0f;
  auto add = [&](float m, float l, const float (&v)[8]) {
    const float t = fmaxf(top, m);
    const float before = top == t ? 1.0f : ex2_approx(top - t);
    const float w = m == t ? 1.0f : ex2_approx(m - t);
    top = t;
    sum = fmaf(w, l, sum * before);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, v[e], acc[e] * before);
  };
  for (int i0 = k; i0 < n; i0 += SJ_LANES * SJ_BATCH) {
    float m[SJ_BATCH], l[SJ_BATCH], v[SJ_BATCH][8];
#pragma unroll
    for (int u = 0; u < SJ_BATCH; ++u)
      if (i0 + SJ_LANES * u < n) read(i0 + SJ_LANES * u, m[u], l[u], v[u]);
#pragma unroll
    for (int u = 0; u < SJ_BATCH; ++u)
      if (i0 + SJ_LANES * u < n) add(m[u], l[u], v[u]);
  }
  const unsigned lanes = ((1u << SJ_LANES) - 1u) << (tid & 31 & ~(SJ_LANES - 1));
#pragma unroll
  for (int d = 1; d < SJ_LANES; d <<= 1) {
    // both of two lanes add the lower one's first: the same bits in both
    float m = __shfl_xor_sync(lanes, top, d), l = __shfl_xor_sync(lanes, sum, d);
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __shfl_xor_sync(lanes, acc[e], d);
    if (k & d) {
      const float mt = top, lt = sum;
      top = m;
      sum = l;
      m = mt;
      l = lt;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = acc[e];
        acc[e] = v[e];
        v[e] = x;
      }
    }
    add(m, l, v);
  }
  if (k != 0) return;
  const float inv = kv_inverse(sum, top != -INFINITY);
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] *= inv;
  kv_store8(a.O, a.o_dtype, token * a.o_ts + head * a.o_hs + col, acc);
}

int64_t up32(int64_t n) { return (n + 31) / 32 * 32; }

// The workspace: the list, the rows' states of both sets, the passes' parts.
struct Layout {
  int64_t list, o[2], ml[2], rec[2], parts[2], total;
};
// Room for either kernel that the rows may want, so that less of anything never needs
// more.
int64_t parts_bytes(int64_t rows, int64_t d, int sms) {
  size_t n = std::max(kv_pass_workspace_bytes(8, d, sms), kv_pass_workspace_bytes(16, d, sms));
  if (kv_pass_unit(rows) == 256) n = std::max(n, kv_pass_workspace_bytes(256, d, sms));
  return static_cast<int64_t>(n);
}
Layout layout_of(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_q,
                 int64_t requests, int64_t groups, int sms) {
  Layout l;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up32(bytes);
    return here;
  };
  const int64_t group = q_heads / kv_heads;
  l.list = take(static_cast<int64_t>(sizeof(KvEntry)) * (requests + groups));
  for (int i = 0; i < 2; ++i) {
    l.o[i] = take(4 * tokens * q_heads * d);
    l.ml[i] = take(8 * tokens * q_heads);
    l.rec[i] = take(16 * tokens * q_heads);
    l.parts[i] = take(parts_bytes((i == 0 ? tokens : max_q) * group, d, sms));
  }
  l.total = at;
  return l;
}

}  // namespace

void kv_set_shared_bytes(int64_t bytes) {
  g_worth.store(bytes < 0 ? SP_WORTH : bytes, std::memory_order_relaxed);
}

size_t kv_attention_shared_workspace_bytes(int64_t tokens, int64_t q_heads, int64_t kv_heads, int64_t d,
                                           int64_t max_q, int64_t requests, int64_t groups) {
  const int sms = kv_sm_count();
  if (sms <= 0 || requests > SP_MAX || groups > SP_MAX) return 0;
  // (16 bytes to bring a workspace that begins at a 16-byte boundary to a 32-byte one)
  return static_cast<size_t>(layout_of(tokens, q_heads, kv_heads, d, max_q, requests, groups, sms).total + 16);
}

cudaError_t launch_kv_attention_shared(const KvAttn& q, const KvGroups& g, cudaStream_t st) {
  const KvCache& c = q.cache;
  const int sms = kv_sm_count();
  const size_t need = kv_attention_shared_workspace_bytes(q.tokens, q.q_heads, c.heads, c.d, q.max_q,
                                                          q.requests, g.n);
  // Without groups or room for the states, or where not even prefixes as long as the table
  // would be worth a pass (groups may be empty: one of all requests spares most), or the
  // requests' rows are many: each request for itself.
  const int64_t most = q.width << kv_page_shift(c.page);
  // (Q may have room for more rows than the requests have)
  const int64_t tokens = std::min(q.tokens, std::max<int64_t>(1, q.max_q) * q.requests);
  const int64_t bytes = 2 * c.heads * c.d, worth = g_worth.load(std::memory_order_relaxed);
  if (g.n == 0 || need == 0 || q.ws == nullptr || q.ws_bytes < need ||
      (worth > 0 && ((q.requests - 1) * most < worth / bytes ||
                     tokens * (q.q_heads / c.heads) > SP_MOST_ROWS * q.requests)))
    return launch_kv_attention(q, st);
  const Layout l = layout_of(q.tokens, q.q_heads, c.heads, c.d, q.max_q, q.requests, g.n, sms);
  char* ws = static_cast<char*>(q.ws) + (reinterpret_cast<uintptr_t>(q.ws) & 16);
  KvEntry* list = reinterpret_cast<KvEntry*>(ws + l.list);
  // Which kernels: one for both where their units are alike, or the group's rows make two of
  // the requests' units at most.
  const int64_t group = q.q_heads / c.heads;
  const int64_t rows = std::max<int64_t>(1, tokens / g.n) * group;
  int prefix_unit = kv_pass_unit(rows);
  const int own_unit = kv_pass_unit(q.max_q * group);
  const bool one = own_unit != 256 && prefix_unit != 256 &&
                   (own_unit == prefix_unit || rows <= 2 * own_unit);
  if (one) prefix_unit = own_unit;
  PlanArgs p{};
  p.lens = q.lens;
  p.cu = q.cu;
  p.groups = g.groups;
  p.shared = g.shared;
  p.table = q.table;
  p.table_stride = q.table_stride;
  p.requests = static_cast<int>(q.requests);
  p.n = static_cast<int>(g.n);
  p.worth = worth / bytes;
  p.capacity = static_cast<int>(most < 0x7FFFFF00 ? most : 0x7FFFFF00);
  p.page_shift = kv_page_shift(c.page);
  p.list = list;
  p.split = !one && prefix_unit == 256 && g.n <= KV_SPLIT_GROUPS;
  p.heads = static_cast<int>(c.heads);
  p.group = static_cast<int>(group);
  p.own_rows = own_unit;
  p.prefix_entry = c.d == 64 ? SP_PREFIX_64 : SP_PREFIX_128;
  p.own_entry = own_unit == 256 ? p.prefix_entry
                                : (own_unit == 8 ? SP_OWN_8 : SP_OWN_16) * (c.d == 64 ? SP_OWN_64 : 1.0f) * (c.fmt == FMT_INT8 ? SP_OWN_INT8 : 1.0f);
  const bool alone = g.n > SP_MANY_GROUPS || q.requests * q.width <= SP_ENTRIES * g.n;
  const int cluster = alone ? 1 : SP_CLUSTER;
  cudaError_t e = launch_early(kv_plan_kernel, dim3(static_cast<unsigned>(cluster), static_cast<unsigned>(g.n)),
                               SP_THREADS, 0, cluster, st, p);
  if (e != cudaSuccess) return e;
  JoinArgs j{};
  JoinSet* sets[2] = {&j.prefix, &j.own};
  for (int i = 0; i < 2; ++i) {
    sets[i]->states.o = reinterpret_cast<float*>(ws + l.o[i]);
    sets[i]->states.ml = reinterpret_cast<float2*>(ws + l.ml[i]);
    sets[i]->states.rec = reinterpret_cast<int4*>(ws + l.rec[i]);
    sets[i]->parts = reinterpret_cast<const float*>(ws + l.parts[i]);
  }
  j.prefix.unit = prefix_unit;
  j.own.unit = own_unit;
  for (int i = 0; i < 2; ++i) sets[i]->ctas = kv_pass_ctas(sets[i]->unit, c.d, sms);
  KvPassArgs pass{};
  pass.prefix = j.prefix.states;
  pass.own = j.own.states;
  pass.groups = list;
  pass.n_groups = p.split ? static_cast<int>(g.n) : 0;
  KvAttn a = q;
  a.window = 0;
  if (one) {
    j.prefix.parts = j.own.parts;
    pass.list = list;
    pass.entries = g.n + q.requests;
  } else {
    pass.list = list;
    pass.entries = g.n;
    a.ws = ws + l.parts[0];
    a.ws_bytes = static_cast<size_t>(kv_pass_workspace_bytes(j.prefix.unit, c.d, sms));
    if ((e = launch_kv_pass(a, pass, j.prefix.unit, true, sms, st)) != cudaSuccess) return e;
    pass.list = list + g.n;
    pass.entries = q.requests;
  }
  a.ws = ws + l.parts[1];
  a.ws_bytes = static_cast<size_t>(kv_pass_workspace_bytes(j.own.unit, c.d, sms));
  if ((e = launch_kv_pass(a, pass, j.own.unit, one, sms, st)) != cudaSuccess) return e;
  j.cu = q.cu;
  j.requests = static_cast<int>(q.requests);
  j.rows = q.tokens * q.q_heads;
  j.q_heads = static_cast<int>(q.q_heads);
  j.O = q.O;
  j.o_dtype = q.o_dtype;
  j.o_ts = q.o_ts;
  j.o_hs = q.o_hs;
  const int lanes = j.rows <= SJ_FEW_ROWS ? 4 : 1;
  const dim3 grid(static_cast<unsigned>((j.rows * (c.d / 8) * lanes + SJ_THREADS - 1) / SJ_THREADS));
  auto kern = c.d == 64 ? (lanes == 4 ? kv_join_states_kernel<64, 4> : kv_join_states_kernel<64, 1>)
                        : (lanes == 4 ? kv_join_states_kernel<128, 4> : kv_join_states_kernel<128, 1>);
  return launch_early(kern, grid, SJ_THREADS, 0, 1, st, j);
}

}  // namespace mxk
