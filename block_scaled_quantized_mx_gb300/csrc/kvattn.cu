// kvattn.cu -- attention over the 8-bit paged key/value cache, for few query
// rows per request (single tokens, drafts).
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
//     stretch of it.  A long request is spread over many CTAs, many short
//     ones share one;
//   * a producer warp walks the stretch: it brings the rows of Q to f16, reads
//     the block table and loads each page's P x d codes with one TMA box
//     (swizzled, so that the reads below are free of bank conflicts), ahead of
//     the consumers; pages that a request does not have are not loaded;
//   * four consumer warps each take a quarter of a tile's keys, with their own
//     running maximum and sum (no barrier per tile): codes become f16 in
//     registers (exact for all three formats) and feed mma.sync m16n8k16 with
//     the keys (S = K Q^T) and then V's columns (O = V^T P) as the 16 rows
//     and the query rows as the 8 columns.  The contraction order is permuted
//     so that a lane's consecutive codes of a key are its share of the
//     operand: K needs no transposition, V a byte permute, P one movmatrix;
//   * page scales never touch the codes: K's multiplies the score, V's goes into
//     the probability's exponent, which as a power of two is exact.
// With rows as the narrow side of the product, eight rows (a group of up to
// eight heads) cost half the products, exponentials and registers of sixteen:
// the kernel comes with 8 rows (three CTAs an SM) and 16 (two CTAs).
//
// Precision.  Q is brought to f16 with a power of two per row (so that its
// largest value is in [1, 2): what f16 drops is 2^-25 of it, as fp32
// accumulation would), scores, sums and outputs accumulate in fp32, and P, with
// V's scale in its exponent (kv_kernel.cuh), is rounded to f16: relative 2^-11 of
// a weight, or 2^-28 of the row's largest product of a weight and a scale (2^-25 of
// P that is 2^3 at least for that product).
//
// A unit cut between CTAs leaves its parts (un-normalised O, maximum, sum) in
// the workspace, and a second, small kernel joins them in a fixed order.  It
// is launched as a programmatic dependent, so that its start-up hides behind
// the first.  (Counting the parts' arrivals in memory and letting the last
// one join them took 27 us after the last tile with 57 CTAs to a unit, 131072
// keys in 8 cache heads: every arrival waited for its turn on the counter,
// and one CTA did all the adding.)  Every wait is bounded.
//
// Measured: 64 requests of 8192 keys (32 heads on 8 cache heads of 128, E4M3)
// 168 us, 6.4 TB/s, 0.94 of the copy rate; one of 131072 keys 50 us, of which
// about 7 are the start and the join; 256 of up to 4096 keys, a head of 64 to
// each cache head, int8, pages of 16, 204 us, 5.3 TB/s.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kv_common.cuh"
#include "kv_kernel.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

__device__ unsigned int g_status_kv = 0;

constexpr int KA_WARPS = 4;                // consumer warps
constexpr int KA_CONS = 32 * KA_WARPS;
constexpr int KA_THREADS = KA_CONS + 32;
// V's scales within 2^3 of each other count as the largest of them in a step: the
// row's largest product is then 2^3 instead of 2^6 at least, still 2^17 above
// the smallest normal f16.
constexpr int KA_ALIKE = 3;
constexpr int KA_RED = 36;                 // floats per row of the staging: 32, padded

// Keys per tile: 16 KB of codes of K and as many of V.  (128 keys of 64 values a
// tile left each warp 32 short keys between two waits.)
template <int D>
constexpr int ka_tk() {
  return D == 64 ? 256 : 128;
}

// CTAs per SM of the 8-row (NR = 1) and the 16-row (NR = 2) kernel.
template <int NR>
constexpr int ka_ctas_per_sm() {
  return NR == 1 ? 3 : 2;
}

// What the producer says about a segment: one CTA's part of a unit.
template <int ROWS>
struct KaSeg {
  int tile, count;             // first key tile, number (0: no more segments)
  int len;                     // the request's length
  int live;                    // rows of the unit that exist
  int all_lo, all_hi;          // keys that every live row sees: no mask needed
  int any_lo, any_hi;          // keys that some row sees
  int part;                    // the unit is shared with other CTAs
  int slot;                    // workspace slot of the part
  alignas(8) float fr[ROWS];   // scale * log2 e * the row's power of two
  int lo[ROWS], hi[ROWS];      // keys [lo, hi) that the row sees
  long long out[ROWS];         // the row's first element of O
};

// A unit that begins in this CTA's stretch and goes on in others': what the
// joining kernel needs (live 0: there is none).
template <int ROWS>
struct KaJoin {
  int live;                    // rows
  int parts;                   // CTAs that share it: this one and the next ones
  int first_slot;              // this CTA's slot; the others use their first
  int pad;
  long long out[ROWS];         // the rows' first elements of O
};

template <int D, int NR>
struct KaSmem {
  static constexpr int ROWS = 8 * NR;
  static constexpr int TK = ka_tk<D>();
  static constexpr int MAX_PAGES = TK / 16;            // pages in a tile
  static constexpr int TILE = TK * D;                  // codes of one tile of K or V
  static constexpr int RING = NR == 1 ? 65536 : 98304;
  static constexpr int STAGES = RING / (2 * TILE);
  // staging of the warps' O: [warp][8 rows][KA_RED]
  static constexpr int RED_OFF = RING;
  static constexpr int RED_BYTES = KA_WARPS * 8 * KA_RED * 4;
  // Q fragments, two slots of [row tile][D / 32][lane] x 16 bytes
  static constexpr int Q_OFF = RED_OFF + RED_BYTES;
  static constexpr int Q_SLOT = NR * (D / 32) * 512;
  static constexpr int SEG_OFF = Q_OFF + 2 * Q_SLOT;
  static constexpr int SEG_BYTES = (sizeof(KaSeg<ROWS>) + 15) / 16 * 16;
  static constexpr int ML_OFF = SEG_OFF + 2 * SEG_BYTES;     // (m, v): [warp][row]; l: [warp][row]
  static constexpr int PG_OFF = ML_OFF + 3 * KA_WARPS * ROWS * 4;
  static constexpr int PG_STAGE = MAX_PAGES * 8;             // per page: K scale, V exponent
  static constexpr int BAR_OFF = PG_OFF + STAGES * PG_STAGE;
  static constexpr int MISC_OFF = BAR_OFF + STAGES * 16 + 32;
  static constexpr int TOTAL = MISC_OFF + 128;
  static constexpr int ALLOC = TOTAL + 1024;
  static_assert(ka_ctas_per_sm<NR>() * (ALLOC + 1024) <= 233472, "CTAs per SM");
};

struct KaArgs {
  KvView v;
  const uint16_t* Q;
  void* O;
  long long q_ts, q_hs, o_ts, o_hs;
  int bf16;
  int o_dtype;
  float scale_log2e;
  float* ws;                   // two slots per CTA: [rows][D] of O, then m[rows], l[rows]
  uint8_t* joins;              // one KaJoin per CTA, behind the slots
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

// a / b for a >= 0, b > 0; 32-bit where both fit, which is several times faster.
__device__ __forceinline__ long long ka_div(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// One request's share of the work list.
struct KaReq {
  KvReq r;
  int tiles;                   // key tiles of each of its units, and one for its overhead
  int tile0;                   // its first tile
  int row_tiles;
  long long units;             // row tiles x cache heads; 0: nothing for this kernel
};

template <int ROWS, int TK>
__device__ __forceinline__ KaReq ka_request(const KaArgs& a, int b) {
  KaReq q;
  q.r = kv_request(a.v, b);
  const long long rows = static_cast<long long>(q.r.n) * a.v.group;
  const int first = kv_first_key(a.v, q.r, 0);
  q.tile0 = first / TK;
  q.tiles = 1 + max(1, (q.r.len + TK - 1) / TK - q.tile0);
  q.row_tiles = static_cast<int>((rows + ROWS - 1) / ROWS);
  q.units = static_cast<long long>(q.row_tiles) * a.v.heads;
  return q;
}

// The walk over one CTA's stretch of the list.  Each unit stands in it with
// its tiles behind one entry more, for the time it takes to begin and end a
// unit (about that of a tile): without it a stretch of many short units took
// 68 us where the median took 43 (48 requests of 0 to 6000 keys, window 2048).
template <int ROWS, int TK>
struct KaWalk {
  long long w, w1;             // next entry of the list, end of the stretch
  long long base;              // first entry of request b
  int b;
  KaReq q;
  // the current segment
  int head, row_tile, tile, count;
  bool begins, ends;
  long long unit_start, unit_end;   // the unit's first tile's entry, its end

  __device__ __forceinline__ bool next(const KaArgs& a) {
    while (w < w1) {
      while (w >= base + q.units * q.tiles) {
        base += q.units * q.tiles;
        if (++b >= a.v.requests) return false;
        q = ka_request<ROWS, TK>(a, b);
      }
      const long long u = ka_div(w - base, q.tiles);
      int t = static_cast<int>((w - base) - u * q.tiles);   // 0: the extra entry
      if (t == 0) {
        t = 1;
        if (++w >= w1) return false;          // the unit's tiles are the next CTA's
      }
      row_tile = static_cast<int>(ka_div(u, a.v.heads));
      head = static_cast<int>(u - static_cast<long long>(row_tile) * a.v.heads);
      unit_start = base + u * q.tiles + 1;
      unit_end = unit_start + q.tiles - 1;
      tile = q.tile0 + t - 1;
      count = static_cast<int>(min(static_cast<long long>(q.tiles - t), w1 - w));
      begins = t == 1;
      ends = t + count == q.tiles;
      w += count;
      return true;
    }
    return false;
  }
};

// movmatrix: the 8 x 8 matrix of 16-bit elements held a row per four lanes,
// transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t r) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(r));
  return d;
}

// The maximum of a row's values over the warp's keys (the lanes of one t).
__device__ __forceinline__ float ka_over_keys(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
}

// All consumer threads' verdict: true if it is true for each of them.
__device__ __forceinline__ bool ka_all(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.and.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "n"(KA_CONS)
      : "memory");
  return r != 0;
}

template <int FMT, int D, int NR>
__global__ void __launch_bounds__(KA_THREADS, ka_ctas_per_sm<NR>())
kv_attention_kernel(const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const KaArgs a) {
  using L = KaSmem<D, NR>;
  constexpr int ROWS = L::ROWS, TK = L::TK, KW = TK / KA_WARPS, KS = KW / 16;
  using Seg = KaSeg<ROWS>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar_full = base + L::BAR_OFF, bar_empty = bar_full + 8 * L::STAGES;
  const uint32_t bar_seg = bar_empty + 8 * L::STAGES, bar_seg_empty = bar_seg + 16;
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + L::MISC_OFF);
  long long* sm_base = reinterpret_cast<long long*>(gbase + L::MISC_OFF + 16);
  long long* sm_scan = reinterpret_cast<long long*>(gbase + L::MISC_OFF + 24);   // [5]
  KaReq* sm_req = reinterpret_cast<KaReq*>(gbase + L::MISC_OFF + 64);
  int* sm_b = reinterpret_cast<int*>(gbase + L::MISC_OFF + 64 + sizeof(KaReq));
  static_assert(sizeof(KaReq) <= 56, "fits");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  if (tid == 0) {
    for (int i = 0; i < L::STAGES; ++i) {
      mbar_init(bar_full + 8 * i, 2);
      mbar_init(bar_empty + 8 * i, KA_WARPS);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_seg + 8 * i, 1);
      mbar_init(bar_seg_empty + 8 * i, KA_WARPS);
    }
    *abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  // ---- the list: its length, and where this CTA's stretch begins
  const int per = (a.v.requests + KA_THREADS - 1) / KA_THREADS;
  const int rb0 = min(a.v.requests, tid * per), rb1 = min(a.v.requests, rb0 + per);
  long long mine = 0;
  KaReq last{};
  for (int b = rb0; b < rb1; ++b) {
    last = ka_request<ROWS, TK>(a, b);
    mine += last.units * last.tiles;
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
  KaJoin<ROWS>* join = reinterpret_cast<KaJoin<ROWS>*>(a.joins) + cta;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (cta >= ctas) {                         // the whole CTA: nothing was started
    if (a.ws != nullptr && tid == 0) join->live = 0;
    return;
  }
  // the first `longer` CTAs take one entry more than the others
  const long long share = ka_div(total, ctas), longer = total - share * ctas;
  const long long w0 = cta * share + min(cta, longer);
  const long long w1 = w0 + share + (cta < longer ? 1 : 0);
  if (w0 >= before && w0 < before + mine) {
    long long p = before;
    for (int b = rb0; b < rb1; ++b) {
      const KaReq q = per == 1 ? last : ka_request<ROWS, TK>(a, b);
      const long long n = q.units * q.tiles;
      if (w0 < p + n) {
        *sm_b = b;
        *sm_req = q;
        *sm_base = p;
        break;
      }
      p += n;
    }
  }
  __syncthreads();

  if (warp == KA_WARPS) {
    // ------------------------------------------------------------ producer
    KaWalk<ROWS, TK> walk;
    walk.b = *sm_b;
    walk.base = *sm_base;
    walk.q = *sm_req;
    walk.w = w0;
    walk.w1 = w1;
    const bool whole = a.ws == nullptr;
    if (whole) {
      // units stay whole: the CTA in whose stretch a unit begins takes all of it
      const long long t = walk.q.tiles;
      walk.w = walk.base + (w0 - walk.base + t - 1) / t * t;   // may be the next request's first
    } else if (lane == 0) {
      join->live = 0;
    }
    const int g = lane >> 2, t4 = lane & 3;
    int it = 0, seg_it = 0;
    bool ok = true, first = true;
    while (ok) {
      bool more;
      if (whole) {
        more = walk.w < w1;
        walk.w1 = 0x7FFFFFFFFFFFFFFFll;
        more = more && walk.next(a);
      } else {
        more = walk.next(a);
      }
      const int ss = seg_it & 1;
      Seg* seg = reinterpret_cast<Seg*>(gbase + L::SEG_OFF + ss * L::SEG_BYTES);
      if (!mbar_wait(bar_seg_empty + 8 * ss, ((seg_it >> 1) & 1) ^ 1, abort)) {
        if (lane == 0) ka_timeout(abort, 0x41);
        ok = false;
        break;
      }
      ++seg_it;
      if (!more) {
        if (lane == 0) {
          seg->count = 0;
          mbar_arrive(bar_seg + 8 * ss);
        }
        break;
      }
      const KvReq rq = walk.q.r;
      const int rows = rq.n * a.v.group;
      const int shift = a.v.page_shift;
      const int per_tile = TK >> shift;
      // the rows' raw values, on their way before anything waits
      uint4 raw_q[NR][D / 32];
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const int r = walk.row_tile * ROWS + 8 * nr + g;
        const bool live = r < rows;
        const int token = live ? r / a.v.group : 0;
        const int qh = walk.head * a.v.group + (live ? r - token * a.v.group : 0);
        const uint16_t* src = a.Q + (rq.q0 + token) * a.q_ts + qh * a.q_hs + t4 * (D / 4);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          raw_q[nr][c] = make_uint4(0, 0, 0, 0);
          if (live) raw_q[nr][c] = *reinterpret_cast<const uint4*>(src + 8 * c);
        }
      }
      const int* row = a.v.table + static_cast<long long>(walk.b) * a.v.table_stride;
      // A tile's pages: the first MAX_PAGES lanes look after their keys, the next
      // after their values.  A page's id is -1 where the request has none and for an id
      // outside the cache (whose keys are NaN).  Ids are read two tiles ahead
      // and scales one, so that no tile waits for either.
      const int slot = lane & (L::MAX_PAGES - 1);
      const bool is_v = (lane & L::MAX_PAGES) != 0;
      const int first_key = kv_first_key(a.v, rq, walk.row_tile * ROWS / a.v.group);
      const uint8_t* scales = is_v ? a.v.v_scales : a.v.k_scales;
      auto page_of = [&](int i) {
        const int key0 = (walk.tile + i) * TK;
        int id = -1;
        if (i < walk.count && lane < 2 * L::MAX_PAGES && slot < per_tile &&
            kv_follows(a.v, rq, first_key, key0 + (slot << shift)))
          id = row[(key0 >> shift) + slot];
        return id < a.v.pages ? id : -1;
      };
      auto scale_of = [&](int id) -> uint32_t {
        return id >= 0 ? scales[static_cast<long long>(id) * a.v.heads + walk.head] : 0xFFu;
      };
      int id0 = page_of(0), id1 = page_of(1);
      uint32_t code = scale_of(id0);
      // loads tile i of the segment
      auto load = [&](int i) {
        const int st = it % L::STAGES;
        const int id2 = page_of(i + 2);
        const uint32_t next_code = scale_of(id1);
        if (!mbar_wait(bar_empty + 8 * st, ((it / L::STAGES) & 1) ^ 1, abort)) {
          if (lane == 0) ka_timeout(abort, 0x42);
          return false;
        }
        const unsigned have = __ballot_sync(0xFFFFFFFFu, id0 >= 0);
        const uint32_t full = bar_full + 8 * st;
        if (lane == 0)
          mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(have)) * (D << shift));
        __syncwarp();
        if (id0 >= 0) {
          const int y =
              static_cast<int>((static_cast<long long>(id0) * a.v.heads + walk.head) << shift);
          tma_load_2d(base + st * 2 * L::TILE + (is_v ? L::TILE : 0) + slot * (D << shift),
                      is_v ? &tmV : &tmK, full, 0, y);
        }
        // K's scale as a factor, NaN where V's is (the two halves of the lanes tell
        // each other); V's as its code, -1 for a page that was not loaded (its
        // codes must not be used)
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, code, L::MAX_PAGES);
        if (lane < 2 * L::MAX_PAGES && slot < per_tile) {
          uint32_t* pg = reinterpret_cast<uint32_t*>(gbase + L::PG_OFF + st * L::PG_STAGE);
          pg[2 * slot + (is_v ? 1 : 0)] =
              is_v ? (id0 >= 0 ? code : 0xFFFFFFFFu)
                   : __float_as_uint(kv_scale_value(other == 0xFFu ? 0xFFu : code));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
        id0 = id1;
        id1 = id2;
        code = next_code;
        ++it;
        return true;
      };
      // the CTA's first tiles are on their way before its first rows are
      // prepared: the ring is empty
      int loaded = 0;
      if (it == 0)
        while (loaded < min(walk.count, L::STAGES) && ok) {
          ok = load(loaded);
          ++loaded;
        }
      if (!ok) break;
      // ---- the rows: what they see, and Q as the B operand's fragments: lane
      // (g, t) holds row g's values [D/4 t, D/4 (t + 1))
      int all_lo = 0, all_hi = 0x7FFFFFFF, any_lo = 0x7FFFFFFF, any_hi = 0;
      long long out_of_lane = 0;
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const int rr = 8 * nr + g, r = walk.row_tile * ROWS + rr;
        const bool live = r < rows;
        const int token = live ? r / a.v.group : 0;
        const int qh = walk.head * a.v.group + (live ? r - token * a.v.group : 0);
        uint32_t w[D / 8];
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 v = raw_q[nr][c];
          w[4 * c] = v.x;
          w[4 * c + 1] = v.y;
          w[4 * c + 2] = v.z;
          w[4 * c + 3] = v.w;
        }
        const int lo = live ? kv_first_key(a.v, rq, token) : 0;
        const int hi = live ? kv_end_key(a.v, rq, token) : 0;
        if (live) {
          all_lo = max(all_lo, lo);
          all_hi = min(all_hi, hi);
          if (hi > lo) {
            any_lo = min(any_lo, lo);
            any_hi = max(any_hi, hi);
          }
        }
        // a power of two that brings the row's largest value into [1, 2)
        float down = 1.0f, up = 1.0f;
        if (a.bf16) {
          uint32_t top = 0;
#pragma unroll
          for (int e = 0; e < D / 8; ++e)
            top = max(top, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          kv_row_factors(top, down, up);
#pragma unroll
          for (int e = 0; e < D / 8; ++e)
            w[e] = cvt_f16x2(__uint_as_float(w[e] << 16) * down,
                             __uint_as_float(w[e] & 0xFFFF0000u) * down);
        }
        uint4* qs = reinterpret_cast<uint4*>(gbase + L::Q_OFF + ss * L::Q_SLOT) +
                    nr * (D / 32) * 32 + lane;
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
          qs[32 * c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
        const long long out = (rq.q0 + token) * a.o_ts + qh * a.o_hs;
        if (t4 == 0) {
          seg->fr[rr] = a.scale_log2e * up;
          seg->lo[rr] = lo;
          seg->hi[rr] = hi;
          seg->out[rr] = out;
        }
        // lane r of the warp keeps row r's
        const long long of = __shfl_sync(0xFFFFFFFFu, out, 4 * (lane & 7));
        if ((lane >> 3) == nr) out_of_lane = of;
      }
      all_lo = __reduce_max_sync(0xFFFFFFFFu, all_lo);
      all_hi = __reduce_min_sync(0xFFFFFFFFu, all_hi);
      any_lo = __reduce_min_sync(0xFFFFFFFFu, any_lo);
      any_hi = __reduce_max_sync(0xFFFFFFFFu, any_hi);
      if (lane == 0) {
        seg->tile = walk.tile;
        seg->count = walk.count;
        seg->len = rq.len;
        seg->live = min(ROWS, rows - walk.row_tile * ROWS);
        seg->all_lo = all_lo;
        seg->all_hi = all_hi;
        seg->any_lo = any_lo;
        seg->any_hi = any_hi;
        seg->part = !(walk.begins && walk.ends);
        // the CTA's first segment and its last can be parts
        seg->slot = static_cast<int>(2 * cta + (first ? 0 : 1));
      }
      // the unit goes on in other CTAs: say what joins it
      if (walk.begins && !walk.ends) {
        if (lane == 0) {
          join->live = min(ROWS, rows - walk.row_tile * ROWS);
          const long long last = walk.unit_end - 1, edge = longer * (share + 1);
          const long long c1 =
              last < edge ? ka_div(last, share + 1) : longer + ka_div(last - edge, share);
          join->parts = static_cast<int>(c1 - cta + 1);
          join->first_slot = static_cast<int>(2 * cta + (first ? 0 : 1));
        }
        if (lane < ROWS) join->out[lane] = out_of_lane;
      }
      first = false;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_seg + 8 * ss);

      for (int i = loaded; i < walk.count && ok; ++i) ok = load(i);
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
  constexpr int STEPS = D / 16;               // 16-value steps of S's contraction
  constexpr int CHUNKS = D / 64;              // 16-byte chunks of a key per lane
  constexpr int MT = D / 16;                  // 16-column tiles of O
  float* red = reinterpret_cast<float*>(gbase + L::RED_OFF);
  float2* sm_mv = reinterpret_cast<float2*>(gbase + L::ML_OFF);
  float* sm_l = reinterpret_cast<float*>(sm_mv + KA_WARPS * ROWS);
  int it = 0, seg_it = 0;
  bool ok = true;
  while (true) {
    const int ss = seg_it & 1;
    if (ok && !mbar_wait(bar_seg + 8 * ss, (seg_it >> 1) & 1, abort)) {
      if (lane == 0) ka_timeout(abort, 0x43);
      ok = false;
    }
    ok = ka_all(ok);
    if (!ok) break;
    ++seg_it;
    const Seg* seg = reinterpret_cast<const Seg*>(gbase + L::SEG_OFF + ss * L::SEG_BYTES);
    const int count = seg->count;
    if (count == 0) break;
    const int tile0 = seg->tile, len = seg->len;
    const int all_lo = seg->all_lo, all_hi = seg->all_hi, any_lo = seg->any_lo, any_hi = seg->any_hi;
    // The lane's rows of S^T are 8 nr + 2 t + e.  B fragments of Q, and the rows'
    // factors: with 16 rows read for each tile, where keeping them cost spills
    // (48 requests of four drafts 56 us, now 51).
    uint32_t qf[NR][D / 8];
    float fr[NR][2];
    auto read_q = [&] {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const uint4* qs = reinterpret_cast<const uint4*>(gbase + L::Q_OFF + ss * L::Q_SLOT) +
                          nr * (D / 32) * 32 + lane;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const uint4 w = qs[32 * c];
          qf[nr][4 * c] = w.x;
          qf[nr][4 * c + 1] = w.y;
          qf[nr][4 * c + 2] = w.z;
          qf[nr][4 * c + 3] = w.w;
        }
      }
    };
    auto read_fr = [&] {
#pragma unroll
      for (int nr = 0; nr < NR; ++nr) {
        const float2 u = *reinterpret_cast<const float2*>(seg->fr + 8 * nr + 2 * t4);
        fr[nr][0] = u.x;
        fr[nr][1] = u.y;
      }
    };
    if constexpr (NR == 1) {
      read_q();
      read_fr();
    }
    float m[NR][2], l[NR][2], v[NR][2];       // v: P's and O's exponent
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[nr][e] = KV_NO_MAX;
        v[nr][e] = KV_NO_V;
        l[nr][e] = 0.0f;
      }
    }
    float o[MT][NR][4];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int nr = 0; nr < NR; ++nr)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nr][e] = 0.0f;
    for (int i = 0; i < count; ++i, ++it) {
      const int st = it % L::STAGES;
      if (ok && !mbar_wait(bar_full + 8 * st, (it / L::STAGES) & 1, abort)) {
        if (lane == 0) ka_timeout(abort, 0x44);
        ok = false;
      }
      ok = __all_sync(0xFFFFFFFFu, ok);
      const int key0 = (tile0 + i) * TK + warp * KW;
      if (ok && key0 < any_hi && key0 + KW > any_lo) {
        const uint32_t kt = base + st * 2 * L::TILE;
        const uint32_t vt = kt + L::TILE;
        const uint2* pg = reinterpret_cast<const uint2*>(gbase + L::PG_OFF + st * L::PG_STAGE);
        const bool masked = key0 < all_lo || key0 + KW > all_hi;
        if constexpr (NR == 2) read_q();
        // ---- scores of the warp's steps of 16 keys: x[.][.][2 h + e] is key g + 8 h
        // and row 2 t + e
        float x[KS][NR][4];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[s][nr][e] = 0.0f;
          const int key = warp * KW + 16 * s + g;   // and key + 8: the same swizzle
#pragma unroll
          for (int c = 0; c < CHUNKS; ++c) {
            const int chunk = CHUNKS * t4 + c;
            const int sw = D == 128 ? (chunk ^ (key & 7)) : (chunk ^ ((key >> 1) & 3));
            const uint4 ka = ld_shared_v4(kt + key * D + sw * 16);
            const uint4 kb = ld_shared_v4(kt + (key + 8) * D + sw * 16);
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t f[4];
              kv_f16_pairs<FMT>(wa[q], f[0], f[2]);
              kv_f16_pairs<FMT>(wb[q], f[1], f[3]);
#pragma unroll
              for (int nr = 0; nr < NR; ++nr)
                mma_16816(x[s][nr], f, qf[nr][2 * (4 * c + q)], qf[nr][2 * (4 * c + q) + 1]);
            }
          }
        }
        // ---- log2 units, mask, running maximum
        int v_top = -1, v_low = 255;
        float mx[NR][2];
        if constexpr (NR == 2) read_fr();
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) mx[nr][0] = mx[nr][1] = -INFINITY;
        uint2 page[KS];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          page[s] = pg[(warp * KW + 16 * s) >> a.v.page_shift];
          if (page[s].y < 0xFFu) {
            v_top = max(v_top, static_cast<int>(page[s].y));
            v_low = min(v_low, static_cast<int>(page[s].y));
          }
#pragma unroll
          for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float f = fr[nr][e] * __uint_as_float(page[s].x);
              float y0 = x[s][nr][e] * f, y1 = x[s][nr][2 + e] * f;
              if (masked) {
                const int lo = seg->lo[8 * nr + 2 * t4 + e], hi = seg->hi[8 * nr + 2 * t4 + e];
                const int j = key0 + 16 * s + g;
                if (j < lo || j >= hi) y0 = -INFINITY;
                if (j + 8 < lo || j + 8 >= hi) y1 = -INFINITY;
              }
              x[s][nr][e] = y0;
              x[s][nr][2 + e] = y1;
              mx[nr][e] = fmaxf(mx[nr][e], fmaxf(y0, y1));
            }
        }
        // v's condition with the step's largest scale, whether a row sees it or not;
        // what it moves to knows better
        bool moves = false;
        float x_top[NR][2];
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            x_top[nr][e] = ka_over_keys(mx[nr][e]);
            const float over = x_top[nr][e] - m[nr][e];
            moves |= over > KV_LAZY || over + (static_cast<float>(v_top) - v[nr][e]) > KV_LAZY;
          }
        if (__any_sync(0xFFFFFFFFu, moves)) {
          const bool alike = v_top - v_low <= KA_ALIKE;
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            float by[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float mn = kv_next_m(m[nr][e], x_top[nr][e]);
              float t = x_top[nr][e] - mn + static_cast<float>(v_top);
              if (!alike) {
                t = -INFINITY;
#pragma unroll
                for (int s = 0; s < KS; ++s)
                  if (page[s].y < 0xFFu)
                    t = fmaxf(t, fmaxf(x[s][nr][e], x[s][nr][2 + e]) - mn +
                                     static_cast<float>(page[s].y));
                t = ka_over_keys(t);
              }
              const float vn = kv_next_v(v[nr][e], m[nr][e] - mn, t);
              by[e] = kv_move_o(m[nr][e], mn, v[nr][e], vn);
              l[nr][e] *= ex2_approx(m[nr][e] - mn);
              m[nr][e] = mn;
              v[nr][e] = vn;
            }
#pragma unroll
            for (int c = 0; c < MT; ++c) {
              o[c][nr][0] *= by[0];
              o[c][nr][1] *= by[1];
              o[c][nr][2] *= by[0];
              o[c][nr][3] *= by[1];
            }
          }
        }
        // ---- probabilities and the product with V, a step of 16 keys at a time
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int code = static_cast<int>(page[s].y);
          const float ve = static_cast<float>(code);
          uint32_t pb[NR][2];
#pragma unroll
          for (int nr = 0; nr < NR; ++nr) {
            float nm[2], back[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float b = kv_p_shift(ve, v[nr][e]);
              nm[e] = b - m[nr][e];
              back[e] = kv_unshift(b);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float q[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                q[e] = ex2_approx(x[s][nr][2 * h + e] + nm[e]);
                if (masked) {
                  const int j = key0 + 16 * s + g + 8 * h;
                  if (j < seg->lo[8 * nr + 2 * t4 + e] || j >= seg->hi[8 * nr + 2 * t4 + e])
                    q[e] = 0.0f;
                }
                l[nr][e] = fmaf(q[e], back[e], l[nr][e]);
              }
              pb[nr][h] = transpose8(cvt_f16x2(q[0], q[1]));
            }
          }
          // codes of keys 2t, 2t + 1, 2t + 8, 2t + 9 of the step; those that
          // were not loaded, or lie behind the request's end, count as zero
          constexpr int W = D / 32;            // 32-bit words of a key per lane
          uint32_t vw[4][W];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = warp * KW + 16 * s + 2 * t4 + (r & 1) + 8 * (r >> 1);
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
          if (code < 0 || key0 + 16 * s + 16 > len) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int j = key0 + 16 * s + 2 * t4 + (r & 1) + 8 * (r >> 1);
              if (code < 0 || j >= len)
#pragma unroll
                for (int e = 0; e < W; ++e) vw[r][e] = 0u;
            }
          }
#pragma unroll
          for (int e = 0; e < W; ++e) {
            // zip two keys' bytes: columns 4e .. 4e + 3 as pairs of keys; two
            // columns make the 16 rows of an operand (lane g: columns of chunk g)
            uint32_t f0[4], f1[4];
            kv_f16_pairs<FMT>(__byte_perm(vw[0][e], vw[1][e], 0x5140), f0[0], f0[1]);
            kv_f16_pairs<FMT>(__byte_perm(vw[2][e], vw[3][e], 0x5140), f0[2], f0[3]);
            kv_f16_pairs<FMT>(__byte_perm(vw[0][e], vw[1][e], 0x7362), f1[0], f1[1]);
            kv_f16_pairs<FMT>(__byte_perm(vw[2][e], vw[3][e], 0x7362), f1[2], f1[3]);
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) {
              mma_16816(o[2 * e][nr], f0, pb[nr][0], pb[nr][1]);
              mma_16816(o[2 * e + 1][nr], f1, pb[nr][0], pb[nr][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_empty + 8 * st);
    }

    // ---- the four warps' results as one
#pragma unroll
    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[nr][e];
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 4);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 8);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 16);
        if (g == 0) {
          sm_mv[warp * ROWS + 8 * nr + 2 * t4 + e] = make_float2(m[nr][e], v[nr][e]);
          sm_l[warp * ROWS + 8 * nr + 2 * t4 + e] = sum;
        }
      }
    kv_bar_sync(1, KA_CONS);
    // the maximum of a row's m over the warps, and of its units 2^v at that m
    auto common = [&](const float2 (&mv)[KA_WARPS], float& M, float& V) {
      M = V = -INFINITY;
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) M = fmaxf(M, mv[w].x);
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) V = fmaxf(V, mv[w].y + (mv[w].x - M));
    };
    // weight of this warp's rows relative to the common references
    float wgt[NR][2];
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      float2 mv[2][KA_WARPS];
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) {
        const float4 u = *reinterpret_cast<const float4*>(sm_mv + w * ROWS + 8 * nr + 2 * t4);
        mv[0][w] = make_float2(u.x, u.y);
        mv[1][w] = make_float2(u.z, u.w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M, V;
        common(mv[e], M, V);
        wgt[nr][e] = kv_move_o(m[nr][e], M, v[nr][e], V);
      }
    }
    const bool part = seg->part;
    const int live = seg->live;
    float* slot = a.ws + static_cast<long long>(seg->slot) * (ROWS * (D + 2));
#pragma unroll
    for (int nr = 0; nr < NR; ++nr) {
      if (8 * nr >= live) break;
      // the row that a thread of the first two warps adds up, and its sum
      const int rr = 8 * nr + ((tid >> 3) & 7), c8 = tid & 7;
      const bool adds = tid < 64 && rr < live;
      float M, V, unit0, unit, lsum = 0.0f;
      float2 mv[KA_WARPS];
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) mv[w] = sm_mv[w * ROWS + rr];
      common(mv, M, V);
      kv_o_unit(V, unit0, unit);
#pragma unroll
      for (int w = 0; w < KA_WARPS; ++w) {
        lsum += sm_l[w * ROWS + rr] * ex2_approx(mv[w].x - M);
      }
      const bool saw = max(seg->lo[rr], seg->tile * TK) < min(seg->hi[rr], (seg->tile + seg->count) * TK);
      if (!part) unit0 *= kv_inverse(lsum, saw);
      if (!saw) M = -INFINITY;
      const long long out = seg->out[rr];
      // rounds over 4 columns of each of the 8 chunks
#pragma unroll
      for (int rd = 0; rd < D / 32; ++rd) {
        if (rd + nr > 0) kv_bar_sync(1, KA_CONS);    // the staging has been read
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float4*>(red + (warp * 8 + 2 * t4 + e) * KA_RED + 4 * g) =
              make_float4(o[2 * rd][nr][e] * wgt[nr][e], o[2 * rd][nr][2 + e] * wgt[nr][e],
                          o[2 * rd + 1][nr][e] * wgt[nr][e], o[2 * rd + 1][nr][2 + e] * wgt[nr][e]);
        kv_bar_sync(1, KA_CONS);
        if (adds) {
          float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < KA_WARPS; ++w) {
            const float4 v =
                *reinterpret_cast<const float4*>(red + (w * 8 + (rr & 7)) * KA_RED + 4 * c8);
            s.x += v.x;
            s.y += v.y;
            s.z += v.z;
            s.w += v.w;
          }
          const int col = (D / 8) * c8 + 4 * rd;
          s.x = s.x * unit0 * unit;
          s.y = s.y * unit0 * unit;
          s.z = s.z * unit0 * unit;
          s.w = s.w * unit0 * unit;
          if (part)
            *reinterpret_cast<float4*>(slot + rr * D + col) = s;
          else
            kv_store4(a.O, a.o_dtype, out + col, s);
        }
      }
      if (part && adds && c8 == 0) {
        slot[ROWS * D + rr] = M;
        slot[ROWS * (D + 1) + rr] = lsum;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_seg_empty + 8 * ss);
  }

}

// Join the parts of the unit that begins in main CTA blockIdx.x's stretch:
// M = max m_p, O = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p.  One block per (unit,
// 32 columns); a thread takes a row and four columns of every groups-th part,
// with the M so far carried along, so that no load waits for a maximum, and
// the groups' sums meet in shared memory, in order.  Latency bounds it: two
// reads in a row, what to join and the parts.  (With the maxima read first, then
// the weights, then the parts, one request of 131072 keys took 54.5 us, now 50.2;
// batches of eight parts 49.2, but 48 requests of four drafts 53.7 instead of
// 52.6; 256 threads, which leave the main kernel's last CTAs less room, 58.)
// Reads of the parts go around L1 (another kernel wrote them).
constexpr int KJ_THREADS = 128;
template <int D, int ROWS>
__global__ void __launch_bounds__(KJ_THREADS)
kv_join_kernel(const float* __restrict__ ws, const KaJoin<ROWS>* joins, void* O, int o_dtype) {
  constexpr int BATCH = 4, GROUPS = 16;
  constexpr long long PART = ROWS * (D + 2);
  __shared__ float sm_m[KJ_THREADS], sm_l[KJ_THREADS];
  __shared__ float4 sm_acc[KJ_THREADS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const KaJoin<ROWS>* join = joins + blockIdx.x;
  const int4 head = __ldcg(reinterpret_cast<const int4*>(join));
  const int live = head.x, n = head.y;
  if (live == 0) return;
  const int tid = threadIdx.x;
  const int items = live * 8;                          // (row, 4 columns)
  const int groups = min(min(KJ_THREADS / items, GROUPS), n);
  const int grp = tid / items;                         // >= groups: no part of the sum
  const int row = (tid - grp * items) >> 3;
  const int col = 32 * blockIdx.y + 4 * (tid & 7);
  const long long out = __ldcg(&join->out[row]);
  const float* first = ws + head.z * PART;
  const float* rest = ws + 2ll * blockIdx.x * PART;    // part p > 0: slot 2 (CTA + p)
  float top = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (grp < groups)
    for (int p0 = grp; p0 < n; p0 += BATCH * groups) {
      float m[BATCH], l[BATCH];
      float4 v[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const int p = p0 + i * groups;
        if (p >= n) break;
        const float* part = p == 0 ? first : rest + 2 * p * PART;
        m[i] = __ldcg(part + ROWS * D + row);
        l[i] = __ldcg(part + ROWS * (D + 1) + row);
        v[i] = ld_global_cg_f4(part + row * D + col);
      }
      float t = top;
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (p0 + i * groups < n) t = fmaxf(t, m[i]);
      const float before = top == t ? 1.0f : ex2_approx(top - t);
      top = t;
      sum *= before;
      acc.x *= before;
      acc.y *= before;
      acc.z *= before;
      acc.w *= before;
#pragma unroll
      for (int i = 0; i < BATCH; ++i)
        if (p0 + i * groups < n) {
          const float w = m[i] == t ? 1.0f : ex2_approx(m[i] - t);
          sum = fmaf(w, l[i], sum);
          acc.x = fmaf(w, v[i].x, acc.x);
          acc.y = fmaf(w, v[i].y, acc.y);
          acc.z = fmaf(w, v[i].z, acc.z);
          acc.w = fmaf(w, v[i].w, acc.w);
        }
    }
  sm_m[tid] = top;
  sm_l[tid] = sum;
  sm_acc[tid] = acc;
  __syncthreads();
  if (tid >= items) return;
  float t = top;
  for (int i = 1; i < groups; ++i) t = fmaxf(t, sm_m[i * items + tid]);
  sum = 0.0f;
  acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int i = 0; i < groups; ++i) {
    const float mi = sm_m[i * items + tid];
    const float w = mi == t ? 1.0f : ex2_approx(mi - t);
    const float4 u = sm_acc[i * items + tid];
    sum = fmaf(w, sm_l[i * items + tid], sum);
    acc.x = fmaf(w, u.x, acc.x);
    acc.y = fmaf(w, u.y, acc.y);
    acc.z = fmaf(w, u.z, acc.z);
    acc.w = fmaf(w, u.w, acc.w);
  }
  const float inv = kv_inverse(sum, t != -INFINITY);
  acc.x *= inv;
  acc.y *= inv;
  acc.z *= inv;
  acc.w *= inv;
  kv_store4(O, o_dtype, out + col, acc);
}

int ka_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n;
}

// The workspace of a launch: two slots per CTA (rows x (d + 2) floats), then
// a KaJoin per CTA.
int64_t ka_slot_bytes(int64_t d, int nr) { return 8 * nr * (d + 2) * 4; }
int ka_ctas(int nr, int sms) { return (nr == 1 ? ka_ctas_per_sm<1>() : ka_ctas_per_sm<2>()) * sms; }
size_t ka_ws_bytes(int64_t d, int nr, int sms) {
  const size_t join = nr == 1 ? sizeof(KaJoin<8>) : sizeof(KaJoin<16>);
  return static_cast<size_t>(ka_ctas(nr, sms)) * (2 * ka_slot_bytes(d, nr) + join);
}

template <int FMT, int D, int NR>
cudaError_t ka_run(const CUtensorMap& tk, const CUtensorMap& tv, const KaArgs& a, int sms,
                   cudaStream_t st) {
  auto kern = kv_attention_kernel<FMT, D, NR>;
  using L = KaSmem<D, NR>;
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  const int ctas = ka_ctas(NR, sms);
  kern<<<ctas, KA_THREADS, L::ALLOC, st>>>(tk, tv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.ws == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas, D / 32);
  cfg.blockDim = dim3(KJ_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_join_kernel<D, 8 * NR>, static_cast<const float*>(a.ws),
                            reinterpret_cast<const KaJoin<8 * NR>*>(a.joins), a.O, a.o_dtype);
}

template <int FMT>
cudaError_t ka_run_f(int64_t d, int nr, const CUtensorMap& tk, const CUtensorMap& tv,
                     const KaArgs& a, int sms, cudaStream_t st) {
  if (d == 64)
    return nr == 1 ? ka_run<FMT, 64, 1>(tk, tv, a, sms, st) : ka_run<FMT, 64, 2>(tk, tv, a, sms, st);
  return nr == 1 ? ka_run<FMT, 128, 1>(tk, tv, a, sms, st) : ka_run<FMT, 128, 2>(tk, tv, a, sms, st);
}

}  // namespace

namespace {

// Which kernel: the one in this file reads a request's keys once per 16 rows of
// a cache head, the prompt kernel once per 256 but with more to set up and a
// longer way from one step to the next.  Measured with 8 cache heads of 128
// values (this kernel with 16 rows a tile against the prompt kernel): 32 rows, 1
// request of 2000 keys 14 against 24 us, of 32000 35 against 45, 16 requests of
// 500 19 against 22, of 6000 76 against 82, 64 of 500 51 against 61, of 6000 259
// against 271; 48 rows, 1 of 32000 44 against 45, 16 of 500 24 against 22, of
// 6000 106 against 82, 64 of 6000 378 against 272.  With 64 values: 32 rows, 8 of
// 16000 69 against 91, 64 of 2000 85 against 102, 48 rows 97 against 94, 118
// against 103.
constexpr int64_t KA_MOST_ROWS = 32;
bool many_rows(int64_t max_q, int64_t group) { return max_q * group > KA_MOST_ROWS; }

}  // namespace

size_t kv_attention_workspace_bytes(int64_t q_heads, int64_t kv_heads, int64_t d, int64_t max_q) {
  const int sms = ka_sm_count();
  const size_t few = std::max(ka_ws_bytes(d, 1, sms), ka_ws_bytes(d, 2, sms));
  return many_rows(max_q, q_heads / kv_heads) ? std::max(few, kv_prompt_workspace_bytes(d, sms)) : few;
}

cudaError_t launch_kv_attention(const KvAttn& q, cudaStream_t st) {
  const KvCache& c = q.cache;
  const int sms = ka_sm_count();
  if (sms <= 0) return cudaErrorInvalidValue;
  if (many_rows(q.max_q, q.q_heads / c.heads) && q.requests <= kv_prompt_max_requests())
    return launch_kv_prompt(q, sms, st);
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
  // eight rows where the rows that one request has for a cache head fit
  const int nr = q.max_q * a.v.group <= 8 ? 1 : 2;
  if (q.ws && q.ws_bytes >= ka_ws_bytes(c.d, nr, sms)) {
    a.ws = static_cast<float*>(q.ws);
    a.joins = static_cast<uint8_t*>(q.ws) + ka_ctas(nr, sms) * 2 * ka_slot_bytes(c.d, nr);
  }
  CUtensorMap tk, tv;
  if (!kv_tensor_map(&tk, c.k, c) || !kv_tensor_map(&tv, c.v, c)) return cudaErrorInvalidValue;
  switch (c.fmt) {
    case FMT_E4M3: return ka_run_f<FMT_E4M3>(c.d, nr, tk, tv, a, sms, st);
    case FMT_E5M2: return ka_run_f<FMT_E5M2>(c.d, nr, tk, tv, a, sms, st);
    default: return ka_run_f<FMT_INT8>(c.d, nr, tk, tv, a, sms, st);
  }
}

unsigned fetch_and_clear_status_kv(cudaError_t* err) {
  unsigned v = 0, z = 0;
  *err = cudaMemcpyFromSymbol(&v, g_status_kv, sizeof(v));
  if (*err == cudaSuccess) *err = cudaMemcpyToSymbol(g_status_kv, &z, sizeof(z));
  return v;
}

}  // namespace mxk
