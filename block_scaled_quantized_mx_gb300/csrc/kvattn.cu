// kvattn.cu -- attention over the 8-bit paged key/value cache.
//
//   x_ij = scale * q_i . k_j,  o_i = sum_j softmax_j(x_ij) v_j
// over the keys j that query i may see (j < length, not behind its own
// position, inside the window), k_j and v_j being codes times their page's
// power-of-two scale; several query heads share a cache head.
//
// Bound for single tokens: HBM, one byte per cached value.  So the kernel is
// a stream over pages that never widens them in memory:
//   * work is cut evenly, not by request: the key tiles of every (request,
//     row tile, cache head) form one list and each CTA takes an equal
//     stretch of it, two CTAs per SM.  A long request is spread over many
//     CTAs, many short ones share one;
//   * a producer warp reads the block table and loads each page's P x d codes
//     with one TMA box (swizzled, so that the reads below are free of bank
//     conflicts), three tiles of 128 keys ahead; pages that a request does
//     not have are not loaded;
//   * four warps each take 32 keys of a tile, with their own running maximum
//     and sum (no barrier per tile): codes become f16 in registers (exact for
//     all three formats) and feed mma.sync m16n8k16, up to 16 rows (tokens x
//     heads of the group) against 8 keys.  The contraction order is permuted
//     so that a lane's 32 consecutive codes of a key are its share of the B
//     operand: no transposition in memory for K, a byte permute for V;
//   * page scales never touch the codes: K's multiplies the score, V's the
//     probability, which as a power of two is exact.
// The scores and the tensor work of 16 rows need a few percent of the tensor
// rate, so mma.sync suffices here; long query runs go to kvprompt.cu.
//
// Precision.  Q is brought to f16 with a power of two per row (so that its
// largest value is in [1, 2): what f16 drops is 2^-25 of it, as fp32
// accumulation would), scores, sums and outputs accumulate in fp32, and P is
// rounded to f16 (relative 2^-11 of each weight at most).  P carries V's scale relative to the largest
// so far: p 2^(7 + s - s_max), at most 2^15 with the exponentials' slack of
// 2^8, so that a page whose values are 2^20 smaller than another's still
// contributes with full precision.
//
// A unit cut between CTAs leaves its parts (un-normalised O, maximum, sum) in
// the workspace; the CTA that completes the unit's count adds them in CTA
// order, so results do not depend on timing.  Every wait is bounded.
#include <cudaTypedefs.h>

#include <atomic>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kv_common.cuh"
#include "kv_kernel.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

__device__ unsigned int g_status_kv = 0;

constexpr int KA_TK = 128;                 // keys per tile
constexpr int KA_WARPS = 4;                // consumer warps
constexpr int KA_KW = KA_TK / KA_WARPS;    // keys of a tile per warp
constexpr int KA_THREADS = 32 * (KA_WARPS + 1);
constexpr int KA_ROWS = 16;                // rows of a unit
constexpr int KA_MAX_PAGES = KA_TK / 16;   // pages in a tile
constexpr float KA_LAZY = 8.0f;            // slack of the exponentials' reference point
constexpr int KA_P_EXP = 7;                // P is scaled by 2^7: at most 2^(7 + 8) in f16

template <int D>
struct KaSmem {
  static constexpr int TILE = KA_TK * D;               // codes of one tile of K or V
  static constexpr int STAGES = 98304 / (2 * TILE);    // 3 (d 128) or 6 (d 64)
  static constexpr int RING = STAGES * 2 * TILE;
  // staging of the warps' O: [warp][row][32 columns]
  static constexpr int RED_OFF = RING;
  static constexpr int RED_BYTES = KA_WARPS * KA_ROWS * 32 * 4;
  static constexpr int ML_OFF = RED_OFF + RED_BYTES;   // m, l, e: [3][warp][row]
  static constexpr int PG_OFF = ML_OFF + 3 * KA_WARPS * KA_ROWS * 4;
  static constexpr int PG_STAGE = KA_MAX_PAGES * 8;    // per page: K scale, V exponent
  static constexpr int BAR_OFF = PG_OFF + STAGES * PG_STAGE;
  static constexpr int MISC_OFF = BAR_OFF + STAGES * 16;
  static constexpr int TOTAL = MISC_OFF + 64;
  static constexpr int ALLOC = TOTAL + 1024;
  static_assert(2 * (ALLOC + 1024) <= 233472, "two CTAs per SM");
};

struct KaArgs {
  KvView v;
  const uint16_t* Q;
  void* O;
  long long q_ts, q_hs, o_ts, o_hs;
  int bf16;
  int o_dtype;
  float scale_log2e;
  int skip_rows;               // requests with more rows than this are another kernel's
  float* ws;                   // parts: [2 CTAs' slots][16 rows][D], then m, l: [slot][2][16]
  unsigned long long* ctr;
  unsigned long long tag;
};

__device__ __forceinline__ void ka_timeout(volatile int* abort, unsigned site) {
  *abort = 1;
  atomicOr(&g_status_kv, STATUS_TIMEOUT | site);
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Count one arrival (see the K-split's counters in the GEMM: tag << 16 |
// count, a word with another tag counts as zero, completion leaves zero).
__device__ __forceinline__ int ka_arrive(unsigned long long* ctr, unsigned long long tag,
                                         int target) {
  unsigned long long v = 0ull;
  for (int i = 0; i < (1 << 16); ++i) {
    const unsigned long long cnt = ((v >> 16) == tag) ? (v & 0xFFFFull) : 0ull;
    const unsigned long long nv =
        (cnt + 1 == static_cast<unsigned long long>(target)) ? 0ull : (tag << 16) | (cnt + 1);
    const unsigned long long old = atomicCAS(ctr, v, nv);
    if (old == v) return static_cast<int>(cnt + 1);
    v = old;
  }
  return -1;
}

// One request's share of the work list.
struct KaReq {
  KvReq r;
  int tiles;                   // key tiles of each of its units
  int tile0;                   // its first tile
  int row_tiles;
  long long units;             // row tiles x cache heads; 0: nothing for this kernel
};

__device__ __forceinline__ KaReq ka_request(const KaArgs& a, int b) {
  KaReq q;
  q.r = kv_request(a.v, b);
  const long long rows = static_cast<long long>(q.r.n) * a.v.group;
  const int first = kv_first_key(a.v, q.r, 0);
  q.tile0 = first / KA_TK;
  q.tiles = max(1, (q.r.len + KA_TK - 1) / KA_TK - q.tile0);
  q.row_tiles = rows > a.skip_rows ? 0 : static_cast<int>((rows + KA_ROWS - 1) / KA_ROWS);
  q.units = static_cast<long long>(q.row_tiles) * a.v.heads;
  return q;
}

// The walk over one CTA's stretch of the list; every role runs it alike.
struct KaWalk {
  long long w, w1;             // next tile of the list, end of the stretch
  long long base;              // first tile of request b
  int b;
  KaReq q;
  // the current segment
  int head, row_tile, tile, count;
  bool begins, ends;
  long long unit_start, unit_end;

  __device__ __forceinline__ bool next(const KaArgs& a) {
    if (w >= w1) return false;
    while (w >= base + q.units * q.tiles) {
      base += q.units * q.tiles;
      if (++b >= a.v.requests) return false;
      q = ka_request(a, b);
    }
    const long long u = (w - base) / q.tiles;
    const int t = static_cast<int>((w - base) - u * q.tiles);
    head = static_cast<int>(u % a.v.heads);
    row_tile = static_cast<int>(u / a.v.heads);
    unit_start = base + u * q.tiles;
    unit_end = unit_start + q.tiles;
    tile = q.tile0 + t;
    count = static_cast<int>(min(static_cast<long long>(q.tiles - t), w1 - w));
    begins = t == 0;
    ends = t + count == q.tiles;
    w += count;
    return true;
  }
};

template <int FMT, int D>
__global__ void __launch_bounds__(KA_THREADS, 2)
kv_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const KaArgs a) {
  using L = KaSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  float* red = reinterpret_cast<float*>(gbase + L::RED_OFF);
  float* sm_m = reinterpret_cast<float*>(gbase + L::ML_OFF);
  float* sm_l = sm_m + KA_WARPS * KA_ROWS;
  int* sm_e = reinterpret_cast<int*>(sm_l + KA_WARPS * KA_ROWS);
  const uint32_t bar_full = base + L::BAR_OFF, bar_empty = bar_full + 8 * L::STAGES;
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + L::MISC_OFF);
  int* sm_flag = reinterpret_cast<int*>(gbase + L::MISC_OFF + 4);
  int* sm_b = reinterpret_cast<int*>(gbase + L::MISC_OFF + 8);
  long long* sm_base = reinterpret_cast<long long*>(gbase + L::MISC_OFF + 16);
  long long* sm_scan = reinterpret_cast<long long*>(gbase + L::MISC_OFF + 24);   // 5 warps
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(bar_full + 8 * i, 2);
      mbar_init(bar_empty + 8 * i, KA_WARPS);
    }
    *abort = 0;
    *sm_b = -1;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  // ---- the list: its length, and where this CTA's stretch begins
  const int per = (a.v.requests + KA_THREADS - 1) / KA_THREADS;
  const int rb0 = min(a.v.requests, tid * per), rb1 = min(a.v.requests, rb0 + per);
  long long mine = 0;
  for (int b = rb0; b < rb1; ++b) {
    const KaReq q = ka_request(a, b);
    mine += q.units * q.tiles;
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += u;
  }
  if (lane == 31) sm_scan[warp] = incl;
  __syncthreads();
  long long total = 0, before = incl - mine;
  for (int i = 0; i <= KA_WARPS; ++i) {
    if (i < warp) before += sm_scan[i];
    total += sm_scan[i];
  }
  const long long ctas = min(static_cast<long long>(gridDim.x), total);
  const long long cta = blockIdx.x;
  if (cta >= ctas) return;                   // the whole CTA: nothing was started
  long long w0 = total * cta / ctas, w1 = total * (cta + 1) / ctas;
  if (w0 >= before && w0 < before + mine) {
    long long p = before;
    for (int b = rb0; b < rb1; ++b) {
      const KaReq q = ka_request(a, b);
      const long long n = q.units * q.tiles;
      if (w0 < p + n) {
        *sm_b = b;
        *sm_base = p;
        break;
      }
      p += n;
    }
  }
  __syncthreads();
  KaWalk walk;
  walk.b = *sm_b;
  walk.base = *sm_base;
  walk.q = ka_request(a, walk.b);
  walk.w = w0;
  walk.w1 = w1;
  if (a.ws == nullptr) {
    // units stay whole: the CTA in whose stretch a unit begins takes all of it
    const long long t = walk.q.tiles;
    const long long lo = walk.base + (w0 - walk.base + t - 1) / t * t;
    walk.w = lo;                             // may be the next request's first
  }

  if (warp == KA_WARPS) {
    // ------------------------------------------------------------ producer
    int it = 0;
    bool ok = true;
    while (ok) {
      if (a.ws == nullptr) {
        if (walk.w >= w1) break;
        walk.w1 = 0x7FFFFFFFFFFFFFFFll;
      }
      if (!walk.next(a)) break;
      const int len = walk.q.r.len, shift = a.v.page_shift;
      const int per_tile = KA_TK >> shift;
      const int* row = a.v.table + static_cast<long long>(walk.b) * a.v.table_stride;
      for (int i = 0; i < walk.count; ++i, ++it) {
        const int st = it % L::STAGES;
        const int key0 = (walk.tile + i) * KA_TK;
        // the tile's pages, one per lane: its id, or -1 where the request has
        // none; -2 for an id outside the cache, which makes the page NaN
        int id = -1;
        if (lane < per_tile && key0 + (lane << shift) < len) {
          id = row[(key0 >> shift) + lane];
          if (id < 0 || id >= a.v.pages) id = -2;
        }
        if (!mbar_wait(bar_empty + 8 * st, ((it / L::STAGES) & 1) ^ 1, abort)) {
          if (lane == 0) ka_timeout(abort, 0x41);
          ok = false;
          break;
        }
        const unsigned have = __ballot_sync(0xFFFFFFFFu, id >= 0);
        const uint32_t full = bar_full + 8 * st;
        if (lane == 0)
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(have)) * 2u * (D << shift));
        __syncwarp();
        if (id >= 0) {
          const uint32_t dst = base + st * 2 * L::TILE + lane * (D << shift);
          const int y = static_cast<int>((static_cast<long long>(id) * a.v.heads + walk.head)
                                         << shift);
          tma_load_2d(dst, &tmK, full, 0, y);
          tma_load_2d(dst + L::TILE, &tmV, full, 0, y);
        }
        if (lane < per_tile) {
          // K's scale as a factor; V's as its code, 0xFF for NaN and -1 for
          // a page that was not loaded (its codes must not be used)
          float kf = __uint_as_float(0x7FC00000u);
          int ve = -1;
          if (id >= 0) {
            const long long unit = static_cast<long long>(id) * a.v.heads + walk.head;
            kf = kv_scale_value(a.v.k_scales[unit]);
            ve = a.v.v_scales[unit];
          }
          uint2* pg = reinterpret_cast<uint2*>(gbase + L::PG_OFF + st * L::PG_STAGE) + lane;
          *pg = make_uint2(__float_as_uint(kf), static_cast<uint32_t>(ve));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
    }
    // the CTA may not retire before its copies have landed
    for (int i = max(0, it - L::STAGES); i < it; ++i) {
      const long long t0 = clock64();
      while (!mbar_try_wait(bar_full + 8 * (i % L::STAGES), (i / L::STAGES) & 1) &&
             clock64() - t0 < MXK_WAIT_LIMIT_CYCLES) {
      }
    }
    return;
  }

  // ------------------------------------------------------------ consumers
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int STEPS = D / 16;               // 16-value steps of the contraction
  constexpr int CHUNKS = D / 64;              // 16-byte chunks of a key per lane
  constexpr int NT = D / 8;                   // output column tiles
  int it = 0;
  bool ok = true;
  const bool whole = a.ws == nullptr;
  while (true) {
    if (whole) {
      if (walk.w >= w1) break;
      walk.w1 = 0x7FFFFFFFFFFFFFFFll;
    }
    const long long seg_w = walk.w;
    if (!walk.next(a)) break;
    const KvReq rq = walk.q.r;
    const int rows = rq.n * a.v.group;        // all rows of the request and cache head
    // ---- this lane's two rows: what they see, and Q as A fragments
    int lo[2], hi[2];
    uint32_t qf[STEPS][4];
    float fr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = walk.row_tile * KA_ROWS + g + 8 * h;
      const bool live = r < rows;
      const int token = live ? r / a.v.group : 0;
      lo[h] = live ? kv_first_key(a.v, rq, token) : 0;
      hi[h] = live ? kv_end_key(a.v, rq, token) : 0;
      const int qh = walk.head * a.v.group + (live ? r - token * a.v.group : 0);
      const uint16_t* src = a.Q + (rq.q0 + token) * a.q_ts + qh * a.q_hs + t4 * (D / 4);
      uint32_t w[D / 8];
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (live) v = *reinterpret_cast<const uint4*>(src + 8 * c);
        w[4 * c] = v.x;
        w[4 * c + 1] = v.y;
        w[4 * c + 2] = v.z;
        w[4 * c + 3] = v.w;
      }
      // a power of two that brings the row's largest value into [1, 2)
      float down = 1.0f, up = 1.0f;
      if (a.bf16) {
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < D / 8; ++e) top = max(top, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
        top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
        kv_row_factors(top, down, up);
#pragma unroll
        for (int e = 0; e < D / 8; ++e)
          w[e] = cvt_f16x2(__uint_as_float(w[e] << 16) * down,
                           __uint_as_float(w[e] & 0xFFFF0000u) * down);
      }
      fr[h] = a.scale_log2e * up;
#pragma unroll
      for (int s = 0; s < STEPS; ++s) {
        qf[s][h] = w[2 * s];
        qf[s][2 + h] = w[2 * s + 1];
      }
    }
    // keys that every live row of the warp sees need no mask
    int all_lo = max(lo[0], lo[1]), all_hi = min(hi[0] ? hi[0] : 0x7FFFFFFF, hi[1] ? hi[1] : 0x7FFFFFFF);
    {
      const int r0 = walk.row_tile * KA_ROWS + g;
      if (r0 < rows && hi[0] == 0) all_hi = 0;
      if (r0 + 8 < rows && hi[1] == 0) all_hi = 0;
    }
    all_lo = __reduce_max_sync(0xFFFFFFFFu, all_lo);
    all_hi = __reduce_min_sync(0xFFFFFFFFu, all_hi);
    const int any_hi = __reduce_max_sync(0xFFFFFFFFu, max(hi[0], hi[1]));
    const int any_lo = __reduce_min_sync(
        0xFFFFFFFFu, min(hi[0] ? lo[0] : 0x7FFFFFFF, hi[1] ? lo[1] : 0x7FFFFFFF));

    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    int ve = 0;                               // V's reference exponent
    for (int i = 0; i < walk.count; ++i, ++it) {
      const int st = it % L::STAGES;
      if (ok && !mbar_wait(bar_full + 8 * st, (it / L::STAGES) & 1, abort)) {
        if (lane == 0) ka_timeout(abort, 0x42);
        ok = false;
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      const int key0 = (walk.tile + i) * KA_TK + warp * KA_KW;
      if (ok && key0 < any_hi && key0 + KA_KW > any_lo) {
        const uint32_t kt = base + st * 2 * L::TILE;
        const uint32_t vt = kt + L::TILE;
        const uint2* pg = reinterpret_cast<const uint2*>(gbase + L::PG_OFF + st * L::PG_STAGE);
        const bool masked = key0 < all_lo || key0 + KA_KW > all_hi;
        // ---- scores: four tiles of 8 keys
        float x[4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
#pragma unroll
          for (int e = 0; e < 4; ++e) x[n][e] = 0.0f;
          const int key = warp * KA_KW + 8 * n + g;   // this lane's key in the tile
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            const int chunk = CHUNKS * t4 + c;
            const int sw = D == 128 ? (chunk ^ (key & 7)) : (chunk ^ ((key >> 1) & 3));
            const uint4 k4 = ld_shared_v4(kt + key * D + sw * 16);
            const uint32_t w[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              uint32_t b0, b1;
              kv_f16_pairs<FMT>(w[s], b0, b1);
              mma_16816(x[n], qf[4 * c + s], b0, b1);
            }
          }
        }
        // ---- log2 units, mask, running maximum
        int vnew = ve;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          const uint2 page = pg[(warp * KA_KW + 8 * n) >> a.v.page_shift];
          const float kf = __uint_as_float(page.x);
          if (page.y < 0xFFu) vnew = max(vnew, static_cast<int>(page.y));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = e >> 1;
            float y = x[n][e] * (fr[h] * kf);
            if (masked) {
              const int j = key0 + 8 * n + 2 * t4 + (e & 1);
              if (j < lo[h] || j >= hi[h]) y = -INFINITY;
            }
            x[n][e] = y;
            mx[h] = fmaxf(mx[h], y);
          }
        }
        bool moved = vnew != ve;
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
          const float mn = mx[h] > m[h] + KA_LAZY ? mx[h] : m[h];
          alpha[h] = mn == m[h] ? 1.0f : ex2_approx(m[h] - mn);
          moved |= mn != m[h];
          m[h] = mn;
          l[h] *= alpha[h];
        }
        if (__any_sync(0xFFFFFFFFu, moved)) {
          const float vf = kv_exp2i(ve - vnew);
          const float f0 = alpha[0] * vf, f1 = alpha[1] * vf;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][0] *= f0;
            o[n][1] *= f0;
            o[n][2] *= f1;
            o[n][3] *= f1;
          }
          ve = vnew;
        }
        // ---- probabilities and the product with V: two steps of 16 keys
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int kk = warp * KA_KW + 16 * s;
          const int code = static_cast<int>(pg[kk >> a.v.page_shift].y);
          const float vf = code == 0xFF || code < 0 ? __uint_as_float(0x7FC00000u)
                                                    : kv_exp2i(KA_P_EXP + code - ve);
          uint32_t pa[4];
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float x0 = x[2 * s + n][2 * h], x1 = x[2 * s + n][2 * h + 1];
              float p0 = ex2_approx(x0 - m[h]), p1 = ex2_approx(x1 - m[h]);
              float q0 = p0 * vf, q1 = p1 * vf;
              if (masked) {
                const int j = key0 + 16 * s + 8 * n + 2 * t4;
                if (j < lo[h] || j >= hi[h]) p0 = q0 = 0.0f;
                if (j + 1 < lo[h] || j + 1 >= hi[h]) p1 = q1 = 0.0f;
              }
              l[h] += p0 + p1;
              pa[2 * n + h] = cvt_f16x2(q0, q1);
            }
          // codes of keys 2t, 2t + 1, 2t + 8, 2t + 9 of the step; those that
          // were not loaded, or lie behind the request's end, count as zero
          constexpr int W = D / 32;            // 32-bit words of a key per lane
          uint32_t vw[4][W];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = kk + 2 * t4 + (r & 1) + 8 * (r >> 1);
            if constexpr (D == 128) {
              const uint4 v = ld_shared_v4(vt + key * D + ((g ^ (key & 7)) << 4));
              vw[r][0] = v.x;
              vw[r][1] = v.y;
              vw[r][2] = v.z;
              vw[r][3] = v.w;
            } else {
              const uint2 v = kv_ld_shared_v2(vt + key * D + (((g >> 1) ^ ((key >> 1) & 3)) << 4) +
                                              8 * (g & 1));
              vw[r][0] = v.x;
              vw[r][1] = v.y;
            }
          }
          if (code < 0 || key0 + 16 * s + 16 > rq.len) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int j = key0 + 16 * s + 2 * t4 + (r & 1) + 8 * (r >> 1);
              if (code < 0 || j >= rq.len)
#pragma unroll
                for (int e = 0; e < W; ++e) vw[r][e] = 0u;
            }
          }
#pragma unroll
          for (int e = 0; e < W; ++e) {
            // zip two keys' bytes: columns 4e .. 4e + 3 as pairs of keys
            uint32_t b0[4], b1[4];
            kv_f16_pairs<FMT>(__byte_perm(vw[0][e], vw[1][e], 0x5140), b0[0], b0[1]);
            kv_f16_pairs<FMT>(__byte_perm(vw[0][e], vw[1][e], 0x7362), b0[2], b0[3]);
            kv_f16_pairs<FMT>(__byte_perm(vw[2][e], vw[3][e], 0x5140), b1[0], b1[1]);
            kv_f16_pairs<FMT>(__byte_perm(vw[2][e], vw[3][e], 0x7362), b1[2], b1[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) mma_16816(o[4 * e + c], pa, b0[c], b1[c]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_empty + 8 * st);
    }

    // ---- the four warps' results as one
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
      l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
      if (t4 == 0) {
        sm_m[warp * KA_ROWS + g + 8 * h] = m[h];
        sm_l[warp * KA_ROWS + g + 8 * h] = l[h];
        sm_e[warp * KA_ROWS + g + 8 * h] = ve;
      }
    }
    kv_bar_sync(1, 32 * KA_WARPS);
    // weight of this warp's two rows relative to the common reference, with
    // O brought to true units in the end: 2^(e - 127 - KA_P_EXP)
    float wgt[2];
    int top_e = 0;
#pragma unroll
    for (int w = 0; w < KA_WARPS; ++w) top_e = max(top_e, sm_e[w * KA_ROWS]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) M = fmaxf(M, sm_m[w * KA_ROWS + g + 8 * h]);
      wgt[h] = (m[h] == M ? 1.0f : ex2_approx(m[h] - M)) * kv_exp2i(ve - top_e);
    }
    // the row this thread adds up, and its sum
    const int rr = tid >> 3;                  // 0..15
    float M = -INFINITY, lsum = 0.0f;
#pragma unroll
    for (int w = 0; w < KA_WARPS; ++w) M = fmaxf(M, sm_m[w * KA_ROWS + rr]);
#pragma unroll
    for (int w = 0; w < KA_WARPS; ++w) {
      const float mw = sm_m[w * KA_ROWS + rr];
      lsum += sm_l[w * KA_ROWS + rr] * (mw == M ? 1.0f : ex2_approx(mw - M));
    }
    const bool part = !(walk.begins && walk.ends);
    const int r = walk.row_tile * KA_ROWS + rr;
    const bool live = r < rows;
    const float inv = lsum == 0.0f ? 0.0f : 1.0f / lsum;
    const int slot = static_cast<int>(2 * cta + (seg_w == w0 ? 0 : 1));
    float* part_o = a.ws + static_cast<long long>(slot) * (KA_ROWS * (D + 2)) + rr * D;
    const int token = live ? r / a.v.group : 0;
    const int qh = walk.head * a.v.group + (live ? r - token * a.v.group : 0);
    const long long out0 = (rq.q0 + token) * a.o_ts + qh * a.o_hs;
    // rounds over 4 (of the lane's D / 4) columns at a time: lane (g, t) holds
    // columns [D/4 t, D/4 (t + 1)), the first half of them in accumulators 0, 2
#pragma unroll
    for (int rd = 0; rd < NT / 4; ++rd) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float4 v;
          v.x = o[4 * rd][2 * h + half] * wgt[h];
          v.y = o[4 * rd + 1][2 * h + half] * wgt[h];
          v.z = o[4 * rd + 2][2 * h + half] * wgt[h];
          v.w = o[4 * rd + 3][2 * h + half] * wgt[h];
          *reinterpret_cast<float4*>(red + (warp * KA_ROWS + g + 8 * h) * 32 + 8 * t4 + 4 * half) = v;
        }
      kv_bar_sync(1, 32 * KA_WARPS);
      float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const int c8 = tid & 7;                 // 4 columns: lane t = c8 / 2, half c8 & 1
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(red + (w * KA_ROWS + rr) * 32 + 4 * c8);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
      if (live) {
        const int col = (D / 4) * (c8 >> 1) + (D / 8) * (c8 & 1) + 4 * rd;
        // to true units: 2^(top_e - 127), and the 2^KA_P_EXP out of P
        const float f = kv_scale_value(static_cast<uint32_t>(top_e));
        s.x = s.x * (1.0f / (1 << KA_P_EXP)) * f;
        s.y = s.y * (1.0f / (1 << KA_P_EXP)) * f;
        s.z = s.z * (1.0f / (1 << KA_P_EXP)) * f;
        s.w = s.w * (1.0f / (1 << KA_P_EXP)) * f;
        if (part) {
          *reinterpret_cast<float4*>(part_o + col) = s;
        } else {
          s.x *= inv;
          s.y *= inv;
          s.z *= inv;
          s.w *= inv;
          kv_store4(a.O, a.o_dtype, out0 + col, s);
        }
      }
      kv_bar_sync(1, 32 * KA_WARPS);
    }
    if (!part) continue;
    float* part_ml = a.ws + static_cast<long long>(slot) * (KA_ROWS * (D + 2)) + KA_ROWS * D;
    if ((tid & 7) == 0) {
      part_ml[rr] = M;
      part_ml[KA_ROWS + rr] = lsum;
    }
    __threadfence();
    kv_bar_sync(1, 32 * KA_WARPS);
    // which CTAs share this unit: stretch c is [total c / ctas, total (c+1) / ctas)
    const long long c0 = ((walk.unit_start + 1) * ctas - 1) / total;
    const long long c1 = (walk.unit_end * ctas - 1) / total;
    if (tid == 0)
      *sm_flag = ka_arrive(a.ctr + c0, a.tag, static_cast<int>(c1 - c0 + 1)) ==
                 static_cast<int>(c1 - c0 + 1);
    kv_bar_sync(1, 32 * KA_WARPS);
    if (!*sm_flag) continue;
    __threadfence();
    // this CTA came last: the parts in CTA order
    if (live) {
      const int c8 = tid & 7;
      const long long first = total * c0 / ctas == walk.unit_start ? 2 * c0 : 2 * c0 + 1;
      auto at = [&](long long c) {
        return a.ws + (c == c0 ? first : 2 * c) * (KA_ROWS * (D + 2));
      };
      float top = -INFINITY;
      for (long long c = c0; c <= c1; ++c) top = fmaxf(top, __ldcg(at(c) + KA_ROWS * D + rr));
      float ls = 0.0f;
      float4 acc[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (long long c = c0; c <= c1; ++c) {
        const float* p = at(c);
        const float mc = __ldcg(p + KA_ROWS * D + rr);
        const float f = mc == top ? 1.0f : ex2_approx(mc - top);
        ls = fmaf(f, __ldcg(p + KA_ROWS * (D + 1) + rr), ls);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          const float4 v = ld_global_cg_f4(p + rr * D + 32 * e + 4 * c8);
          acc[e].x = fmaf(f, v.x, acc[e].x);
          acc[e].y = fmaf(f, v.y, acc[e].y);
          acc[e].z = fmaf(f, v.z, acc[e].z);
          acc[e].w = fmaf(f, v.w, acc[e].w);
        }
      }
      const float fin = ls == 0.0f ? 0.0f : 1.0f / ls;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        float4 v = acc[e];
        v.x *= fin;
        v.y *= fin;
        v.z *= fin;
        v.w *= fin;
        kv_store4(a.O, a.o_dtype, out0 + 32 * e + 4 * c8, v);
      }
    }
  }
}

int ka_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

constexpr int64_t part_bytes(int64_t d) { return KA_ROWS * (d + 2) * 4; }

// Two slots per CTA, then a counter per CTA.
size_t ka_ws_bytes(int64_t d, int64_t ctas) {
  return static_cast<size_t>(ctas * 2 * part_bytes(d) + ctas * 8);
}

template <int FMT, int D>
cudaError_t ka_run(const CUtensorMap& tk, const CUtensorMap& tv, const KaArgs& a, int ctas,
                   cudaStream_t st) {
  auto kern = kv_attention_kernel<FMT, D>;
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, KaSmem<D>::ALLOC);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  kern<<<ctas, KA_THREADS, KaSmem<D>::ALLOC, st>>>(tk, tv, a);
  return cudaGetLastError();
}

template <int FMT>
cudaError_t ka_run_d(int64_t d, const CUtensorMap& tk, const CUtensorMap& tv, const KaArgs& a,
                     int ctas, cudaStream_t st) {
  return d == 64 ? ka_run<FMT, 64>(tk, tv, a, ctas, st) : ka_run<FMT, 128>(tk, tv, a, ctas, st);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_q) {
  return ka_ws_bytes(d, 2 * ka_sm_count());
}

cudaError_t launch_kv_attention(const KvAttn& q, cudaStream_t st) {
  const KvCache& c = q.cache;
  KaArgs a{};
  a.v = kv_view(q);
  a.Q = static_cast<const uint16_t*>(q.Q);
  a.O = q.O;
  a.q_ts = q.q_ts;
  a.q_hs = q.q_hs;
  a.o_ts = q.o_ts;
  a.o_hs = q.o_hs;
  a.bf16 = q.dtype == DT_BF16;
  a.o_dtype = q.o_dtype;
  a.scale_log2e = q.scale * 1.4426950408889634f;
  a.skip_rows = 0x7FFFFFFF;
  const int ctas = 2 * ka_sm_count();
  if (ctas <= 0) return cudaErrorInvalidValue;
  if (q.ws && q.ws_bytes >= ka_ws_bytes(c.d, ctas)) {
    a.ws = static_cast<float*>(q.ws);
    a.ctr = reinterpret_cast<unsigned long long*>(static_cast<char*>(q.ws) +
                                                  ctas * 2 * part_bytes(c.d));
    a.tag = next_split_tag();
  }
  CUtensorMap tk, tv;
  if (!kv_tensor_map(&tk, c.k, c) || !kv_tensor_map(&tv, c.v, c)) return cudaErrorInvalidValue;
  switch (c.fmt) {
    case FMT_E4M3: return ka_run_d<FMT_E4M3>(c.d, tk, tv, a, ctas, st);
    case FMT_E5M2: return ka_run_d<FMT_E5M2>(c.d, tk, tv, a, ctas, st);
    default: return ka_run_d<FMT_INT8>(c.d, tk, tv, a, ctas, st);
  }
}

unsigned fetch_and_clear_status_kv(cudaError_t* err) {
  unsigned v = 0, z = 0;
  *err = cudaMemcpyFromSymbol(&v, g_status_kv, sizeof(v));
  if (*err == cudaSuccess) *err = cudaMemcpyToSymbol(g_status_kv, &z, sizeof(z));
  return v;
}

}  // namespace mxk
