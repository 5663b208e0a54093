// kvprompt.cu -- attention over the 8-bit paged key/value cache for many query
// rows per request (prompts and their chunks): the formula, the masks and the
// precision of kvattn.cu, on the fifth-generation tensor core.
//
// Bound: the 16-bit tensor rate, 4 d flop per row and visible key.  One CTA
// per SM; a unit is 256 rows of one request and cache head (row r is token
// r / group, head r % group of the group, so that all heads of a group share
// the converted keys), in two tiles of 128 that take turns on the tensor core
// as in attention.cu.  What differs from dense attention:
//   * K and V come as codes.  Warp 0 reads the block table and the scales and
//     loads the codes of blocks of 128 keys page by page with TMA, a block ahead
//     (d 128; three for d 64); four warps turn them into f16 -- exactly, for all three
//     formats -- and write the swizzled operand tiles, two deep each.  The
//     conversion of a block serves both tiles and, through the rows' order, all
//     heads of the group.  (Read from global memory straight into the
//     converting warps' registers, a tile ahead, 64 requests with 128 rows over
//     6000 keys took 352 us against 331.)
//   * page scales stay out of the operands: K's is a factor of the scores of
//     its 16 .. 128 keys, applied with the softmax scale in the exponent's FMA;
//     V's, a power of two, is added to the exponent relative to the row's own
//     reference (kv_kernel.cuh), so P carries it exactly and the row sums take
//     it out again;
//   * rows are converted once per unit: the thread that owns a row brings it
//     to f16 with a power of two of its own, and keeps its mask bounds.  The next
//     unit's go to shared memory before this unit's O is read and written, so
//     that its first scores are under way meanwhile (231 us -> 227);
//   * the units are cut evenly over the SMs, as in kvattn.cu: a stretch of the
//     list of all (request, row tile, cache head, key block)s per CTA, each
//     unit standing with some entries more for what it costs to begin and end
//     one; parts of units go to the workspace and a second kernel joins them.
//   * scores go 64 keys at a time into two buffers per tile, so that a tile's
//     next scores do not wait for its softmax, and each tile has an issuing warp
//     of its own: one warp spends ~850 clocks on the waits and instructions of a
//     tile's step, the tensor core ~620 (one buffer and one warp, with Q in
//     tensor memory: 237 us against 231; two buffers and one warp: 248; one
//     buffer of 128 keys: 240).
// A 2048-token chunk over 8192 keys (32 heads on 8 cache heads of 128) takes
// 217 us, 0.58 of the measured bf16 rate.  Of these the join takes ~11 and
// beginning and ending units ~20; a block of 128 keys for both tiles ~3700
// clocks, where its products alone need 2480 (in steps of 64 keys a product of
// Q K^T takes 48 clocks, not 32).  With no conversion and no exponentials it
// would still be ~3300: hand-offs between the roles.
// Tensor memory, tile t: its score buffers (then P) in columns [256 t, 256 t + 64)
// and [256 t + 64, 256 t + 128), O in [256 t + 128, 256 t + 128 + d).
// Ordering: an issuing warp issues P V of step h before the scores of step h + 2,
// and a commit covers every earlier operation of its thread: once those scores
// are complete so is that product.  Every mbarrier wait is bounded.
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

__device__ unsigned int g_status_kvp = 0;

constexpr int KP_BQ = 128;                 // rows per tile
constexpr int KP_ROWS = 2 * KP_BQ;         // rows of a unit
constexpr int KP_BK = 128;                 // keys per block
constexpr int KP_HK = 64;                  // keys per step of the softmax, two to a block
constexpr int KP_THREADS = 512;            // pages and issuers, two softmax warpgroups, conversion
constexpr int KP_WARPS = KP_THREADS / 32;
// Registers: launched at 128; 72 * 128 + 176 * 256 + 88 * 128 = 65536.
constexpr int KP_REGS_LOW = 72;            // warpgroup 0
constexpr int KP_REGS_SOFT = 176;          // warpgroups 1 and 2
constexpr int KP_REGS_CONV = 88;           // warpgroup 3
constexpr int KP_TMEM_COLS = 512;
// Entries of a unit besides its blocks: with 1, 2, 4 and 8 eight ragged chunks
// took 80, 68, 65 and 72 us when the 2048-token chunk took 242, 239, 237 and 241
// (now 219 with 2, 3, 4 and 6 alike).
constexpr int KP_OVER = 4;
constexpr int KP_PG = 8;                   // blocks whose page data is kept
constexpr int KP_STAGES = 2;               // f16 tiles of K, and of V
constexpr int KP_MAX_REQUESTS = 16384;

// One block: the scales of each 16 of its keys, and what there is of it.
struct KpPages {
  struct {
    float kf;                              // K's scale; NaN where K's or V's is NaN or no page is
    float ve;                              // V's scale code; 0 there
  } of[8];
  float top;                               // the largest ve; -1: no block at all
  int valid;                               // keys of the block in front of the request's end
  int more;                                // another block follows
  int gone;                                // a bit for each 16 keys whose page was not loaded
};

// One CTA's part of a unit, as every role sees it.
struct KpSeg {
  int count;                               // key blocks (0: no more segments)
  int block;                               // the first
  int len;                                 // the request's length
  int n;                                   // its tokens
  long long q0;                            // its first row of Q
  int row0;                                // the unit's first row
  int head;
  int slot;                                // workspace slot, -1: not a part
  int pad;
};

// A unit that begins in this CTA's stretch and goes on in others'.
struct KpJoin {
  int live;                                // rows (0: there is none)
  int parts;                               // CTAs that share it
  int first_slot;                          // this CTA's slot; the others use their first
  int head;
  int row0;
  int pad;
  long long q0;
};

// The key blocks of row tile rt of a request: [first, first + count).
__device__ __forceinline__ int kp_blocks(const KvView& v, const KvReq& r, int rt, int& first) {
  const int rows = r.n * v.group;
  const int t0 = rt * KP_ROWS / v.group;
  const int t1 = (min(rows, (rt + 1) * KP_ROWS) - 1) / v.group;
  const int lo = kv_first_key(v, r, t0), hi = kv_end_key(v, r, t1);
  first = lo / KP_BK;
  const int n = hi > lo ? (hi + KP_BK - 1) / KP_BK - first : 0;
  return n > 0 ? n : 1;
}
__device__ __forceinline__ int kp_row_tiles(const KvView& v, const KvReq& r) {
  return (r.n * v.group + KP_ROWS - 1) / KP_ROWS;
}

// The walk over one CTA's stretch of the list: groups of units (request, row
// tile), in each the cache heads, each with KP_OVER entries and its blocks.
struct KpWalk {
  long long w, w1;
  long long base;              // first entry of the group
  int b, rt, tiles;            // request, row tile, the request's row tiles
  int blocks, block0;          // of each unit of the group
  KvReq r;
  int head, block, count;
  bool begins, ends;
  long long unit_start, unit_end;

  __device__ __forceinline__ void enter(const KvView& v) {   // b, rt -> the rest
    r = kv_request(v, b);
    tiles = kp_row_tiles(v, r);
    if (rt < tiles) blocks = kp_blocks(v, r, rt, block0);
  }
  __device__ __forceinline__ bool next(const KvView& v) {
    while (w < w1) {
      while (w >= base + static_cast<long long>(v.heads) * (KP_OVER + blocks)) {
        base += static_cast<long long>(v.heads) * (KP_OVER + blocks);
        if (++rt < tiles) {
          blocks = kp_blocks(v, r, rt, block0);
          continue;
        }
        rt = 0;
        do {
          if (++b >= v.requests) return false;
          enter(v);
        } while (tiles == 0);
      }
      const int c = KP_OVER + blocks;
      head = static_cast<int>((w - base) / c);
      const long long unit = base + static_cast<long long>(head) * c;
      unit_start = unit + KP_OVER;
      unit_end = unit + c;
      if (w < unit_start) {
        w = unit_start;
        if (w >= w1) return false;           // the unit's blocks are the next CTA's
      }
      const int t = static_cast<int>(w - unit_start);
      block = block0 + t;
      count = static_cast<int>(min(static_cast<long long>(blocks - t), w1 - w));
      begins = t == 0;
      ends = t + count == blocks;
      w += count;
      return true;
    }
    return false;
  }
};

template <int D>
struct KpSmem {
  static constexpr int REGION = 128 * 128;
  static constexpr int Q_BYTES = (D / 64) * REGION;
  static constexpr int K_BYTES = (D / 64) * REGION;       // V's tiles are alike
  static constexpr int V_BYTES = K_BYTES;
  static constexpr int RAW = D == 64 ? 6 : 2;             // tiles of codes, K and V in turn
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + 2 * Q_BYTES;
  static constexpr int V_OFF = K_OFF + KP_STAGES * K_BYTES;
  static constexpr int RAW_BYTES = KP_BK * D;
  static constexpr int RAW_OFF = V_OFF + KP_STAGES * V_BYTES;
  static constexpr int PG_OFF = RAW_OFF + RAW * RAW_BYTES;
  static constexpr int SEG_OFF = PG_OFF + KP_PG * static_cast<int>(sizeof(KpPages));
  static constexpr int BAR_OFF = SEG_OFF + 2 * static_cast<int>(sizeof(KpSeg));
  // k_full, v_full, k_empty, v_empty [stages]; q_full, o_done [tile],
  // s_full, p_full [tile][buffer]; seg_full[2], seg_empty[2], pg_full[8], pg_empty[8];
  // raw_full, raw_empty [RAW]
  static constexpr int BARS = 4 * KP_STAGES + 12 + 4 + 2 * KP_PG + 2 * RAW;
  static constexpr int MISC_OFF = BAR_OFF + BARS * 8;
  static constexpr int WALK_OFF = MISC_OFF + 16;
  static constexpr int TOTAL = WALK_OFF + static_cast<int>(sizeof(KpWalk));
  static constexpr int ALLOC = TOTAL + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
  static_assert(PG_OFF >= KP_MAX_REQUESTS * 4, "the plan's array fits in the operand tiles");
};

struct KpArgs {
  KvView v;
  const uint16_t* Q;
  void* O;
  long long q_ts, q_hs, o_ts, o_hs;
  int bf16;
  int o_dtype;
  float scale_log2e;
  float* ws;                               // two slots per CTA: O as [D / 8][256 rows][8], m[256], l[256];
                                           // 32-byte aligned
  KpJoin* joins;                           // one per CTA
};

__device__ __forceinline__ void kp_timeout(volatile int* abort, unsigned site) {
  *abort = 1;
  atomicOr(&g_status_kvp, STATUS_TIMEOUT | site);
}

// kind::f16 instruction descriptor: D f32, A and B f16, A K-major, B K-major
// (b_mn = 0) or MN-major (1), N >> 3 at bit 17, M = 128.
__device__ __forceinline__ uint32_t kp_idesc(uint32_t n, uint32_t b_mn) {
  return (1u << 4) | (b_mn << 16) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// Whole products in one statement each.  An issuing warp runs them with all 32
// lanes, so that the descriptors stay warp-uniform, and one elected lane
// issues; the election and the predicates are made once per product, and of
// the descriptors only the low words (start addresses) move.  Issued one by
// one, with an election each, the instructions around them took longer than
// the products.
//
// S = Q K^T: D / 16 steps of 16 along rows of 128-byte regions 16 KB apart.
template <int D>
__device__ __forceinline__ void kp_issue_s(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
  const uint32_t a0 = static_cast<uint32_t>(a), a1 = static_cast<uint32_t>(a >> 32);
  const uint32_t b0 = static_cast<uint32_t>(b), b1 = static_cast<uint32_t>(b >> 32);
  asm volatile(
      "{\n\t.reg .pred e, no, yes;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 no, 0, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
      "add.u32 x, %1, 0;\n\tadd.u32 y, %3, 0;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, no;\n\t"
      "add.u32 x, %1, 2;\n\tadd.u32 y, %3, 2;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, yes;\n\t"
      "add.u32 x, %1, 4;\n\tadd.u32 y, %3, 4;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, yes;\n\t"
      "add.u32 x, %1, 6;\n\tadd.u32 y, %3, 6;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, yes;\n\t"
      "}" ::"r"(d), "r"(a0), "r"(a1), "r"(b0), "r"(b1), "r"(id)
      : "memory");
  if constexpr (D == 128)
    asm volatile(
        "{\n\t.reg .pred e, yes;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
      "add.u32 x, %1, 1024;\n\tadd.u32 y, %3, 1024;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, yes;\n\t"
      "add.u32 x, %1, 1026;\n\tadd.u32 y, %3, 1026;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, yes;\n\t"
      "add.u32 x, %1, 1028;\n\tadd.u32 y, %3, 1028;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, yes;\n\t"
      "add.u32 x, %1, 1030;\n\tadd.u32 y, %3, 1030;\n\tmov.b64 da, {x, %2};\n\tmov.b64 db, {y, %4};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %5, yes;\n\t"
        "}" ::"r"(d), "r"(a0), "r"(a1), "r"(b0), "r"(b1), "r"(id)
        : "memory");
}
// O += P V over 64 keys: four steps, P in tensor memory, V's rows 2 KB apart
// per step; acc 0: O is overwritten.
__device__ __forceinline__ void kp_issue_pv(uint32_t d, uint32_t p, uint64_t b, uint32_t id,
                                            uint32_t acc) {
  const uint32_t b0 = static_cast<uint32_t>(b), b1 = static_cast<uint32_t>(b >> 32);
  asm volatile(
      "{\n\t.reg .pred e, first, yes;\n\t.reg .b32 x, y;\n\t.reg .b64 db;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 first, %5, 0;\n\tsetp.eq.b32 yes, 0, 0;\n\t"
      "add.u32 x, %1, 0;\n\tadd.u32 y, %2, 0;\n\tmov.b64 db, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %4, first;\n\t"
      "add.u32 x, %1, 8;\n\tadd.u32 y, %2, 128;\n\tmov.b64 db, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %4, yes;\n\t"
      "add.u32 x, %1, 16;\n\tadd.u32 y, %2, 256;\n\tmov.b64 db, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %4, yes;\n\t"
      "add.u32 x, %1, 24;\n\tadd.u32 y, %2, 384;\n\tmov.b64 db, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %4, yes;\n\t"
      "}" ::"r"(d), "r"(p), "r"(b0), "r"(b1), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void kp_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          bar)
      : "memory");
}

__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Exclusive prefix sum over the block's threads, and the total.
__device__ __forceinline__ long long kp_scan(long long v, long long* sm, long long& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long s = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, s, d);
    if (lane >= d) s += u;
  }
  if (lane == 31) sm[warp] = s;
  __syncthreads();
  long long before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < KP_WARPS; ++w) {
    if (w < warp) before += sm[w];
    all += sm[w];
  }
  __syncthreads();
  return before + s - v;
}

template <int FMT, int D>
__global__ void __launch_bounds__(KP_THREADS, 1)
kv_prompt_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const KpArgs a) {
  using L = KpSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bar_k = base + L::BAR_OFF;
  const uint32_t bar_v = bar_k + 8 * KP_STAGES;
  const uint32_t bar_k_empty = bar_v + 8 * KP_STAGES;
  const uint32_t bar_v_empty = bar_k_empty + 8 * KP_STAGES;
  const uint32_t bar_q = bar_v_empty + 8 * KP_STAGES;
  const uint32_t bar_o_done = bar_q + 16;
  const uint32_t bar_s_full = bar_o_done + 16;
  const uint32_t bar_p_full = bar_s_full + 32;
  const uint32_t bar_seg = bar_p_full + 32;
  const uint32_t bar_seg_empty = bar_seg + 16;
  const uint32_t bar_pg = bar_seg_empty + 16;      // [KP_PG]
  const uint32_t bar_pg_empty = bar_pg + 8 * KP_PG;
  const uint32_t bar_raw = bar_pg_empty + 8 * KP_PG;
  const uint32_t bar_raw_empty = bar_raw + 8 * L::RAW;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + L::MISC_OFF);
  volatile int* abort = reinterpret_cast<volatile int*>(gbase + L::MISC_OFF + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the list: row tiles of each request, then entries of each row tile
  // (in the operand regions, which nothing uses yet)
  KpWalk* walk = reinterpret_cast<KpWalk*>(gbase + L::WALK_OFF);   // warp 0's, kept by lane 0
  long long total, w0, ctas;
  {
    int* sm_rt = reinterpret_cast<int*>(gbase);                        // requests + 1
    long long* sm_scan = reinterpret_cast<long long*>(gbase + L::PG_OFF);
    const int B = a.v.requests;
    const KvTileList list(a.v.tokens, a.v.group, KP_ROWS, B);
    const int per = (B + KP_THREADS - 1) / KP_THREADS;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long mine = 0, tiles;
    for (int b = b0; b < b1; ++b) mine += kp_row_tiles(a.v, kv_request(a.v, b));
    long long at = kp_scan(mine, sm_scan, tiles);
    for (int b = b0; b < b1; ++b) {
      sm_rt[b] = list.start(at);
      at += kp_row_tiles(a.v, kv_request(a.v, b));
    }
    tiles = list.clip(tiles);
    __syncthreads();
    const long long tper = (tiles + KP_THREADS - 1) / KP_THREADS;
    const long long f0 = min(tiles, tid * tper), f1 = min(tiles, f0 + tper);
    // walks the row tiles [f0, f1): calls f(b, rt, request) for each
    auto each = [&](auto f) {
      if (f0 >= f1) return;
      int b = KvTileList::request(sm_rt, B, f0);
      KvReq r = kv_request(a.v, b);
      int rt = static_cast<int>(f0 - sm_rt[b]), n = kp_row_tiles(a.v, r);
      for (long long i = f0; i < f1; ++i, ++rt) {
        while (rt >= n) {
          rt = 0;
          r = kv_request(a.v, ++b);
          n = kp_row_tiles(a.v, r);
        }
        if (!f(b, rt, r)) return;
      }
    };
    mine = 0;
    each([&](int, int rt, const KvReq& r) {
      int first;
      mine += static_cast<long long>(a.v.heads) * (KP_OVER + kp_blocks(a.v, r, rt, first));
      return true;
    });
    long long before = kp_scan(mine, sm_scan, total);
    ctas = min(static_cast<long long>(gridDim.x), total);
    w0 = total * blockIdx.x / max(1ll, ctas);
    if (blockIdx.x < ctas && w0 >= before && w0 < before + mine) {
      long long p = before;
      each([&](int b, int rt, const KvReq& r) {
        int first;
        const int blocks = kp_blocks(a.v, r, rt, first);
        const long long n = static_cast<long long>(a.v.heads) * (KP_OVER + blocks);
        if (w0 >= p + n) {
          p += n;
          return true;
        }
        KpWalk k;
        k.w = w0;
        k.w1 = total * (blockIdx.x + 1) / ctas;
        k.base = p;
        k.b = b;
        k.rt = rt;
        k.enter(a.v);
        if (a.ws == nullptr) {
          // units stay whole: the CTA in whose stretch a unit begins takes all of it
          const long long c = KP_OVER + k.blocks;
          k.w = p + (w0 - p + c - 1) / c * c;          // may be the next group's first
        }
        *walk = k;
        return false;
      });
    }
    __syncthreads();
    KpJoin* join = a.joins ? a.joins + blockIdx.x : nullptr;
    if (tid == 0 && join) join->live = 0;
    if (blockIdx.x >= ctas) return;          // the whole CTA: nothing was started
  }
  // the regions go to their owners, TMA and the tensor core among them
  fence_proxy_async_smem();
  __syncthreads();

  if (tid == 0) {
    for (int i = 0; i < KP_STAGES; ++i) {
      mbar_init(bar_k + 8 * i, 4);
      mbar_init(bar_v + 8 * i, 4);
      mbar_init(bar_k_empty + 8 * i, 2);
      mbar_init(bar_v_empty + 8 * i, 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q + 8 * i, 4);
      mbar_init(bar_o_done + 8 * i, 1);
      mbar_init(bar_s_full + 16 * i, 1);
      mbar_init(bar_s_full + 16 * i + 8, 1);
      mbar_init(bar_p_full + 16 * i, 4);
      mbar_init(bar_p_full + 16 * i + 8, 4);
      mbar_init(bar_seg + 8 * i, 1);
      mbar_init(bar_seg_empty + 8 * i, 10);
    }
    for (int i = 0; i < KP_PG; ++i) {
      mbar_init(bar_pg + 8 * i, 1);
      mbar_init(bar_pg_empty + 8 * i, 12);
    }
    for (int i = 0; i < L::RAW; ++i) {
      mbar_init(bar_raw + 8 * i, 1);
      mbar_init(bar_raw_empty + 8 * i, 4);
    }
    *abort = 0;
    fence_mbar_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == 1) tmem_alloc_cg<1>(smem_u32(tmem_slot), KP_TMEM_COLS);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const KpSeg* segs = reinterpret_cast<const KpSeg*>(gbase + L::SEG_OFF);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(KP_REGS_LOW));
    if (warp == 0) {
      // ------------------------------------------------- segments and pages
      int bt = 0, seg_out = 0, raw_it = 0;
      bool ok = true, first_seg = true, held = false;
      KpPages* pages = reinterpret_cast<KpPages*>(gbase + L::PG_OFF);
      // a block's data stay back until it is known whether another follows
      auto release = [&](int more) {
        if (!held) return;
        const int ps = (bt - 1) & (KP_PG - 1);
        if (lane == 0) {
          pages[ps].more = more;
          mbar_arrive(bar_pg + 8 * ps);
        }
        held = false;
      };
      while (ok) {
        const int ss = seg_out & 1;
        int found = 0;
        if (lane == 0) {
          if (a.ws != nullptr) {
            found = walk->next(a.v);
          } else if (walk->w < walk->w1) {
            const long long w1 = walk->w1;
            walk->w1 = 0x7FFFFFFFFFFFFFFFll;
            found = walk->next(a.v);
            walk->w1 = w1;
          }
        }
        __syncwarp();
        found = __shfl_sync(0xFFFFFFFFu, found, 0);
        release(found);
        if (!found && bt == 0 && lane == 0) {
          // a stretch without blocks: the converting warps wait for the first
          pages[0].top = -1.0f;
          mbar_arrive(bar_pg);
        }
        if (!mbar_wait(bar_seg_empty + 8 * ss, ((seg_out >> 1) & 1) ^ 1, abort)) {
          if (lane == 0) kp_timeout(abort, 0x51);
          break;
        }
        if (lane == 0) {
          KpSeg* s = const_cast<KpSeg*>(segs) + ss;
          s->count = found ? walk->count : 0;
          if (found) {
            s->block = walk->block;
            s->len = walk->r.len;
            s->n = walk->r.n;
            s->q0 = walk->r.q0;
            s->row0 = walk->rt * KP_ROWS;
            s->head = walk->head;
            const int slot = 2 * static_cast<int>(blockIdx.x) + (first_seg ? 0 : 1);
            s->slot = walk->begins && walk->ends ? -1 : slot;
            if (walk->begins && !walk->ends) {
              KpJoin* j = a.joins + blockIdx.x;
              j->live = min(KP_ROWS, walk->r.n * a.v.group - walk->rt * KP_ROWS);
              j->parts = static_cast<int>((walk->unit_end * ctas - 1) / total - blockIdx.x + 1);
              j->first_slot = slot;
              j->head = walk->head;
              j->row0 = walk->rt * KP_ROWS;
              j->q0 = walk->r.q0;
            }
          }
          mbar_arrive(bar_seg + 8 * ss);
        }
        ++seg_out;
        first_seg = false;
        if (!found) break;
        const int count = walk->count, block0 = walk->block, head = walk->head;
        const KvReq rq = walk->r;
        const int* row = a.v.table + static_cast<long long>(walk->b) * a.v.table_stride;
        const int shift = a.v.page_shift;
        const int first_key = kv_first_key(a.v, rq, walk->rt * KP_ROWS / a.v.group);
        __syncwarp();                          // all lanes have read the walk
        // the page of 16 keys, one per lane; -1: none, or outside the cache
        auto page_of = [&](int j) {
          const int key = (block0 + j) * KP_BK + 16 * lane;
          const bool follows = j < count && lane < 8 && kv_follows(a.v, rq, first_key, key);
          const int id = follows ? row[key >> shift] : -1;
          return id < a.v.pages ? id : -1;
        };
        // Ids are read two blocks ahead and scales one: nothing here waits for either.
        int id1 = page_of(0), id2 = page_of(1);
        uint32_t kc1 = 0xFFu, vc1 = 0xFFu;
        auto scales_of = [&](int id) {
          kc1 = vc1 = 0xFFu;
          if (id >= 0) {
            const long long unit = static_cast<long long>(id) * a.v.heads + head;
            kc1 = a.v.k_scales[unit];
            vc1 = a.v.v_scales[unit];
          }
        };
        scales_of(id1);
        for (int j = 0; j < count; ++j) {
          const int id = id1;
          const uint32_t kc = kc1, vc = vc1;
          id1 = id2;
          id2 = page_of(j + 2);
          scales_of(id1);
          const long long unit = id >= 0 ? static_cast<long long>(id) * a.v.heads + head : 0;
          float kf = __uint_as_float(0x7FC00000u);
          float ve = 0.0f;
          if (kc != 0xFFu && vc != 0xFFu) {
            kf = kv_scale_value(kc);
            ve = static_cast<float>(vc);
          }
          const int ps = bt & (KP_PG - 1);
          if (!mbar_wait(bar_pg_empty + 8 * ps, ((bt / KP_PG) & 1) ^ 1, abort)) {
            if (lane == 0) kp_timeout(abort, 0x52);
            ok = false;
            break;
          }
          if (lane < 8) {
            pages[ps].of[lane].kf = kf;
            pages[ps].of[lane].ve = ve;
          }
          const float top = static_cast<float>(__reduce_max_sync(0xFFFFFFFFu, static_cast<int>(ve)));
          const unsigned gone = __ballot_sync(0xFFFFFFFFu, lane < 8 && id < 0);
          if (lane == 0) {
            pages[ps].gone = static_cast<int>(gone);
            pages[ps].top = top;
            pages[ps].valid = rq.len - (block0 + j) * KP_BK;
          }
          __syncwarp();
          ++bt;
          held = true;
          if (j + 1 < count) release(1);       // (of the last one: when the next segment is known)
          // the codes: a box per page, by the lane of its first 16 keys
          const bool loads = id >= 0 && ((16 * lane) & ((1 << shift) - 1)) == 0;
          const unsigned boxes = __popc(__ballot_sync(0xFFFFFFFFu, loads));
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int slot = raw_it % L::RAW;
            if (!mbar_wait(bar_raw_empty + 8 * slot, ((raw_it / L::RAW) & 1) ^ 1, abort)) {
              if (lane == 0) kp_timeout(abort, 0x5e);
              ok = false;
              break;
            }
            const uint32_t full = bar_raw + 8 * slot;
            if (lane == 0) mbar_arrive_expect_tx(full, boxes * (D << shift));
            __syncwarp();
            if (loads)
              tma_load_2d(base + L::RAW_OFF + slot * L::RAW_BYTES + 16 * lane * D,
                          kv ? &tmV : &tmK, full, 0, static_cast<int>(unit << shift));
            ++raw_it;
          }
          if (!ok) break;
        }
      }
      // the CTA may not retire before its copies have landed
      for (int i = max(0, raw_it - L::RAW); i < raw_it; ++i) {
        const long long t0 = clock64();
        while (!mbar_try_wait(bar_raw + 8 * (i % L::RAW), (i / L::RAW) & 1) &&
               clock64() - t0 < MXK_WAIT_LIMIT_CYCLES) {
        }
      }
    } else if (warp <= 2) {
      // ------------------------------------------------- MMA issuer of tile t
      const int t = warp - 1;
      const uint32_t id_qk = kp_idesc(KP_HK, 0);
      const uint32_t id_pv = kp_idesc(D, 1);
      const uint64_t dq = smem_desc(base + L::Q_OFF + t * L::Q_BYTES, 16, 1024, 2);
      const uint64_t dk0 = smem_desc(base + L::K_OFF, 16, 1024, 2);
      const uint64_t dv0 = smem_desc(base + L::V_OFF, L::REGION, 1024, 2);
      const uint32_t s_full = bar_s_full + 16 * t, p_full = bar_p_full + 16 * t;
      int bt = 0, seg_it = 0, own = 0, own_b = 0;   // blocks, units; units and blocks of the tile
      bool ok = true;
      while (ok) {
        const int ss = seg_it & 1;
        if (!mbar_wait(bar_seg + 8 * ss, (seg_it >> 1) & 1, abort)) {
          kp_timeout(abort, 0x56);
          break;
        }
        const int nkb = segs[ss].count;
        if (nkb == 0) break;
        // tile 1 sits a unit of up to 128 rows out: it only hands the blocks back
        const bool works = segs[ss].n * a.v.group - segs[ss].row0 > KP_BQ * t;
        ++seg_it;
        if (works) {
          if (!mbar_wait(bar_q + 8 * t, own & 1, abort)) {
            kp_timeout(abort, 0x57);
            break;
          }
          ++own;
          tc_fence_after();
        }
        // step h: P_h V_h, then the scores of step h + 2 into the same buffer.  The
        // commit behind the two says that both are done: scores h + 2 complete,
        // and O with P_h V_h in it (which is all that the last two say, the very
        // last at its own barrier: the next unit's scores may follow at once).
        const int steps = 2 * nkb;
#pragma unroll 1
        for (int h = -2; h < steps; ++h) {
          const int n = h + 2, buf = h & 1;
          const int gv = bt + (h >> 1), gk = bt + (n >> 1);
          const int sv = gv % KP_STAGES, sk = gk % KP_STAGES;
          const uint32_t s_t = tmem_base + 256 * t + KP_HK * buf;
          if (h >= 0) {
            if (!buf) ok = mbar_wait(bar_v + 8 * sv, (gv / KP_STAGES) & 1, abort);
            if (works) {
              ok = ok && mbar_wait(p_full + 8 * buf, (own_b + (h >> 1)) & 1, abort);
              if (!ok) break;
              tc_fence_after();
              kp_issue_pv(tmem_base + 256 * t + 128, s_t,
                          dv0 + static_cast<uint64_t>((sv * L::V_BYTES + buf * 8192) >> 4), id_pv,
                          h > 0 ? 1u : 0u);
            }
          }
          if (n < steps) {
            if (!buf) ok = ok && mbar_wait(bar_k + 8 * sk, (gk / KP_STAGES) & 1, abort);
            if (!ok) break;
            if (works) {
              tc_fence_after();
              kp_issue_s<D>(s_t, dq,
                            dk0 + static_cast<uint64_t>((sk * L::K_BYTES + buf * 8192) >> 4), id_qk);
            }
          }
          if (works && n <= steps) kp_commit(s_full + 8 * buf);
          if (buf) {
            if (works) {
              if (h >= 0) kp_commit(bar_v_empty + 8 * sv);
              if (n < steps) kp_commit(bar_k_empty + 8 * sk);
            } else if (lane == 0) {
              if (h >= 0) mbar_arrive(bar_v_empty + 8 * sv);
              if (n < steps) mbar_arrive(bar_k_empty + 8 * sk);
            }
          }
          // O's word comes last: who has heard it may leave
          if (works && n > steps) kp_commit(bar_o_done + 8 * t);
        }
        if (!ok) kp_timeout(abort, 0x58);
        bt += nkb;
        if (works) own_b += nkb;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_seg_empty + 8 * ss);
      }
    }
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(KP_REGS_CONV));
    // ------------------------------------------------------------ conversion
    // A step is 512 bytes of codes (4 rows of 128 or 8 of 64), 16 codes a
    // lane; warp ci takes steps ci, ci + 4, ..: all its steps start at the
    // same row mod 8, and each lies within 16 keys.  For d 128 eight
    // consecutive lanes take the four lower chunks of one row and the four
    // upper ones of the next, which keeps the swizzled writes (two 16-byte
    // chunks of f16 a lane) free of bank conflicts.
    const int ci = warp - 12;
    constexpr int SROWS = 512 / D;
    constexpr int IT = KP_BK / SROWS / 4;
    int rl, c;                               // row in the step, chunk of the row
    if constexpr (D == 128) {
      rl = 2 * (lane >> 4) + (((lane >> 2) ^ (lane >> 3)) & 1);
      c = lane & 7;
    } else {
      rl = lane >> 2;
      c = lane & 3;
    }
    const int r0 = ci * SROWS + rl;          // the lane's row in the warp's first step
    const uint32_t to = (c >> 2) * L::REGION + r0 * 128 + (((2 * (c & 3)) ^ (r0 & 7)) << 4);
    const uint32_t from = r0 * D + ((D == 128 ? (c ^ (r0 & 7)) : (c ^ ((r0 >> 1) & 3))) << 4);
    const KpPages* pages = reinterpret_cast<const KpPages*>(gbase + L::PG_OFF);
    // a block's data, once they are there
    auto pages_of = [&](int b) -> const KpPages* {
      if (!mbar_wait(bar_pg + 8 * (b & (KP_PG - 1)), (b / KP_PG) & 1, abort)) {
        if (lane == 0) kp_timeout(abort, 0x53);
        return nullptr;
      }
      return pages + (b & (KP_PG - 1));
    };
    const KpPages* pg = pages_of(0);
    if (pg && pg->top < 0.0f) pg = nullptr;  // there are none
    // tiles in the order K, V of each block
#pragma unroll 1
    for (int tile = 0; pg; ++tile) {
      const int kv = tile & 1, bt = tile >> 1, st = bt % KP_STAGES, slot = tile % L::RAW;
      if (!mbar_wait(bar_raw + 8 * slot, (tile / L::RAW) & 1, abort)) {
        if (lane == 0) kp_timeout(abort, 0x5f);
        break;
      }
      uint4 w[IT];
#pragma unroll
      for (int i = 0; i < IT; ++i)
        w[i] = ld_shared_v4(base + L::RAW_OFF + slot * L::RAW_BYTES + from + i * 2048);
      // keys of V behind the request's end or in pages that were not loaded
      // count as zeros, whatever stands there
      if (kv && (pg->valid < KP_BK || pg->gone)) {
#pragma unroll
        for (int i = 0; i < IT; ++i) {
          const int r = i * 4 * SROWS + r0;
          if (r >= pg->valid || ((pg->gone >> (r >> 4)) & 1)) w[i] = make_uint4(0, 0, 0, 0);
        }
      }
      if (!mbar_wait((kv ? bar_v_empty : bar_k_empty) + 8 * st, ((bt / KP_STAGES) & 1) ^ 1, abort)) {
        if (lane == 0) kp_timeout(abort, 0x54);
        break;
      }
      const uint32_t dst = base + (kv ? L::V_OFF : L::K_OFF) + st * L::K_BYTES + to;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        uint32_t f[8];
        kv_f16_pairs<FMT>(w[i].x, f[0], f[1]);
        kv_f16_pairs<FMT>(w[i].y, f[2], f[3]);
        kv_f16_pairs<FMT>(w[i].z, f[4], f[5]);
        kv_f16_pairs<FMT>(w[i].w, f[6], f[7]);
        const uint32_t p = dst + i * (4 * SROWS * 128);
        st_shared_v4(p, f[0], f[1], f[2], f[3]);
        st_shared_v4(p ^ 16, f[4], f[5], f[6], f[7]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive((kv ? bar_v : bar_k) + 8 * st);
        // only now, with the codes converted and so in registers beyond doubt:
        // arrived right behind the loads, the next copy could overtake them
        mbar_arrive(bar_raw_empty + 8 * slot);
      }
      if (kv) {
        const bool more = pg->more != 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_pg_empty + 8 * (bt & (KP_PG - 1)));
        pg = more ? pages_of(bt + 1) : nullptr;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(KP_REGS_SOFT));
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int urow = KP_BQ * t + 32 * quarter + lane;       // row in the unit
    const uint32_t lane_addr = tmem_base + (static_cast<uint32_t>(32 * quarter) << 16) + 256 * t;
    // blocks; the tile's own units and, per score buffer, its steps; all units
    int bt = 0, own_seg = 0, own0 = 0, own1 = 0, seg_it = 0;
    const uint32_t s_full = bar_s_full + 16 * t;
    bool ok = true, live = false, works = false;
    int lo = 0, hi = 0, count = 0, key00 = 0;
    float fr = 0.0f, m = KV_NO_MAX, l = 0.0f;
    float v = KV_NO_V;                         // P's and O's exponent: kv_kernel.cuh
    while (true) {
      // ---- the next unit's rows, before this unit's are written: its first
      // scores are on their way meanwhile.  (Q is free: the last scores are done.)
      const int ss = seg_it & 1;
      if (!mbar_wait(bar_seg + 8 * ss, (seg_it >> 1) & 1, abort)) {
        if (lane == 0) kp_timeout(abort, 0x5b);
        break;
      }
      const int next_count = segs[ss].count;
      const bool next_works = next_count != 0 && segs[ss].n * a.v.group - segs[ss].row0 > KP_BQ * t;
      bool next_live = false;
      int next_lo = 0, next_hi = 0;
      float up = 1.0f;
      if (next_count != 0) {
        // this thread's row: Q to f16, its bounds and factor
        KvReq rq;
        rq.q0 = segs[ss].q0;
        rq.n = segs[ss].n;
        rq.len = segs[ss].len;
        const int row = segs[ss].row0 + urow;
        next_live = row < rq.n * a.v.group;
        const int token = next_live ? row / a.v.group : 0;
        const int qh = segs[ss].head * a.v.group + (next_live ? row - token * a.v.group : 0);
        next_lo = next_live ? kv_first_key(a.v, rq, token) : 0;
        next_hi = next_live ? kv_end_key(a.v, rq, token) : 0;
        if (next_works) {
          uint32_t w[D / 2];
          const uint16_t* src = a.Q + (rq.q0 + token) * a.q_ts + qh * a.q_hs;
#pragma unroll
          for (int c = 0; c < D / 8; ++c) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (next_live) v = *reinterpret_cast<const uint4*>(src + 8 * c);
            w[4 * c] = v.x;
            w[4 * c + 1] = v.y;
            w[4 * c + 2] = v.z;
            w[4 * c + 3] = v.w;
          }
          if (a.bf16) {
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < D / 2; ++e)
              top = max(top, max((w[e] << 16) & 0x7FFFFFFFu, w[e] & 0x7FFF0000u));
            float down;
            kv_row_factors(top, down, up);
            if (a.scale_log2e < 0.0f) down = -down;
#pragma unroll
            for (int e = 0; e < D / 2; ++e)
              w[e] = cvt_f16x2(__uint_as_float(w[e] << 16) * down,
                               __uint_as_float(w[e] & 0xFFFF0000u) * down);
          } else if (a.scale_log2e < 0.0f) {
#pragma unroll
            for (int e = 0; e < D / 2; ++e) w[e] ^= 0x80008000u;
          }
          const int r = 32 * quarter + lane;
#pragma unroll
          for (int c = 0; c < D / 8; ++c)
            st_shared_v4(base + L::Q_OFF + t * L::Q_BYTES + (c >> 3) * L::REGION + r * 128 +
                             (((c & 7) ^ (r & 7)) << 4),
                         w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_q + 8 * t);
        }
      }
      // ---- this unit's rows (none before the first unit)
      if (works) {
        if (!mbar_wait(bar_o_done + 8 * t, own_seg & 1, abort)) {
          if (lane == 0) kp_timeout(abort, 0x5d);
          break;
        }
        ++own_seg;
        tc_fence_after();
        // a row that saw keys and adds up to nothing had only scores of -infinity
        const bool saw = max(lo, key00) < min(hi, key00 + KP_BK * count);
        float unit0, unit;
        kv_o_unit(v, unit0, unit);
        // (read again rather than kept in registers over the blocks)
        const volatile KpSeg* sg = segs + (ss ^ 1);
        float* part = sg->slot >= 0 ? a.ws + static_cast<long long>(sg->slot) * (KP_ROWS * (D + 2)) : nullptr;
        const int row = sg->row0 + urow, token = row / a.v.group;
        const long long out =
            (sg->q0 + token) * a.o_ts + (sg->head * a.v.group + row - token * a.v.group) * a.o_hs;
        // rows of O 32 bytes at a time where they are that aligned
        const bool by32 = ((reinterpret_cast<uintptr_t>(a.O) |
                            static_cast<uintptr_t>(out * (a.o_dtype == DT_F32 ? 4 : 2))) & 31) == 0;
        const float f = part ? unit0 : unit0 * kv_inverse(l, saw);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(lane_addr + 128 + 32 * c, o);
          tmem_wait_ld();
          if (!live) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f * unit);
          if (part) {
            // lanes hold consecutive rows: whole lines of [8 columns][row][column]
#pragma unroll
            for (int e = 0; e < 4; ++e)
              st_global_v8(part + ((4 * c + e) * KP_ROWS + urow) * 8,
                           *reinterpret_cast<const uint32_t(*)[8]>(o + 8 * e));
          } else if (a.o_dtype == DT_F32) {
            float* dst = static_cast<float*>(a.O) + out + 32 * c;
#pragma unroll
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4*>(dst)[e] =
                  make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          } else {
            uint16_t* dst = static_cast<uint16_t*>(a.O) + out + 32 * c;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float x0 = __uint_as_float(o[16 * h + 2 * e]);
                const float x1 = __uint_as_float(o[16 * h + 2 * e + 1]);
                w[e] = a.o_dtype == DT_BF16 ? cvt_bf16x2(x0, x1) : cvt_f16x2(x0, x1);
              }
              if (by32) {
                st_global_v8(dst + 16 * h, w);
              } else {
                reinterpret_cast<uint4*>(dst + 16 * h)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4*>(dst + 16 * h)[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          }
        }
        if (part && live) {
          part[KP_ROWS * D + urow] = saw ? m : -INFINITY;
          part[KP_ROWS * (D + 1) + urow] = l;
        }
        tc_fence_before();
      }
      if (seg_it > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_seg_empty + 8 * (ss ^ 1));
      }
      ++seg_it;
      if (next_count == 0) break;
      live = next_live;
      works = next_works;
      lo = next_lo;
      hi = next_hi;
      count = next_count;
      key00 = segs[ss].block * KP_BK;
      // a negative scale has gone into Q: the factor of a score is never negative
      fr = fabsf(a.scale_log2e) * up;
      // keys that every live row of this warp sees
      const int all_lo = __reduce_max_sync(0xFFFFFFFFu, live ? lo : 0);
      const int all_hi = __reduce_min_sync(0xFFFFFFFFu, live ? hi : 0x7FFFFFFF);

      m = KV_NO_MAX;
      l = 0.0f;
      v = KV_NO_V;
#pragma unroll 1
      for (int h = 0; h < 2 * count; ++h) {
        const int g = bt + (h >> 1), ps = g & (KP_PG - 1);
        const int key0 = key00 + KP_HK * h;
        if (!mbar_wait(bar_pg + 8 * ps, (g / KP_PG) & 1, abort) ||
            (works && !mbar_wait(s_full + 8 * (h & 1), ((h & 1 ? own1 : own0) + (h >> 1)) & 1, abort))) {
          if (lane == 0) kp_timeout(abort, 0x5c);
          ok = false;
          break;
        }
        if (!works) {                          // the tile has no rows: only say so
          if (lane == 0 && (h & 1)) mbar_arrive(bar_pg_empty + 8 * ps);
          continue;
        }
        tc_fence_after();
        const KpPages* pg = reinterpret_cast<const KpPages*>(gbase + L::PG_OFF) + ps;
        const int p0 = 4 * (h & 1);            // the step's first 16 keys in the block
        uint32_t x0[32], x1[32];
        const uint32_t s_at = lane_addr + KP_HK * (h & 1);
        tmem_ld_32x32b_x32(s_at, x0);
        tmem_ld_32x32b_x32(s_at + 32, x1);
        tmem_wait_ld();
        // Row maximum: of the raw scores of each 16 keys, times their factor.
        // A step that some row does not see whole is scaled and masked first:
        // what is hidden may stand in a page whose factor is NaN.
        const bool masked = key0 < all_lo || key0 + KP_HK > all_hi;
        float f[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) f[p] = fr * pg->of[p0 + p].kf;
        if (masked) {
#pragma unroll
          for (int e = 0; e < KP_HK; ++e) {
            uint32_t& x = e < 32 ? x0[e & 31] : x1[e & 31];
            const float y = __uint_as_float(x) * f[e >> 4];
            x = key0 + e >= lo && key0 + e < hi ? __float_as_uint(y) : 0xFF800000u;   // -inf
          }
#pragma unroll
          for (int p = 0; p < 4; ++p) f[p] = 1.0f;
        }
        float mx = -INFINITY, gx[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const uint32_t(&x)[32] = p < 2 ? x0 : x1;
          float g0 = -INFINITY, g1 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const int i = 16 * (p & 1) + e;
            g0 = max3(g0, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
            g1 = max3(g1, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
          }
          gx[p] = fmaxf(g0, g1) * f[p];
          mx = fmaxf(mx, gx[p]);
        }
        // v's condition with the block's largest scale, whether the row sees it or
        // not; what it moves to knows better
        const float over = mx - m;
        if (__any_sync(0xFFFFFFFFu, over > KV_LAZY || over + (pg->top - v) > KV_LAZY)) {
          const float m_new = kv_next_m(m, mx);
          float tv = -INFINITY;
#pragma unroll
          for (int p = 0; p < 4; ++p) tv = fmaxf(tv, (gx[p] - m_new) + pg->of[p0 + p].ve);
          const float v_new = kv_next_v(v, m - m_new, tv);
          if (h >= 1 && __any_sync(0xFFFFFFFFu, m_new != m || v_new != v)) {
            // the product that last wrote O, of the step before, is done when the
            // next step's scores are
            if (!mbar_wait(s_full + 8 * (~h & 1), ((h & 1 ? own0 : own1) + ((h + 1) >> 1)) & 1, abort)) {
              if (lane == 0) kp_timeout(abort, 0x5a);
              ok = false;
              break;
            }
            tc_fence_after();
            const float by = kv_move_o(m, m_new, v, v_new);
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(lane_addr + 128 + 32 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * by);
              tmem_st_32x32b_x32(lane_addr + 128 + 32 * c, o);
            }
          }
          l *= ex2_approx(m - m_new);
          m = m_new;
          v = v_new;
        }
        // p' = 2^(x - m + b), b = 7 + (V's exponent - v), rounded
        // to f16 and written back over the scores; the sum takes b out again.
        // Hidden scores are -inf and stay it: b and m are finite.
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t(&x)[32] = c ? x1 : x0;
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int p = 2 * c + q;
            const float b = kv_p_shift(pg->of[p0 + p].ve, v);
            const float nm = b - m;
            const uint64_t f2 = pack2(f[p], f[p]), nm2 = pack2(nm, nm);
            uint64_t sum = pack2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float y0, y1;
              unpack2(fma2(pack2(__uint_as_float(x[16 * q + 2 * e]),
                                 __uint_as_float(x[16 * q + 2 * e + 1])),
                           f2, nm2),
                      y0, y1);
              const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
              pk[8 * q + e] = cvt_f16x2(e0, e1);
              sum = add2(sum, pack2(e0, e1));
            }
            float a0, a1;
            unpack2(sum, a0, a1);
            l = fmaf(a0 + a1, kv_unshift(b), l);
          }
          tmem_st_32x32b_x16(s_at + 16 * c, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_p_full + 16 * t + 8 * (h & 1));
          if (h & 1) mbar_arrive(bar_pg_empty + 8 * ps);
        }
      }
      bt += count;
      if (!ok) break;
      if (works) {
        // the phase behind the last scores of buffer 0, before the next unit's
        if (!mbar_wait(s_full, (own0 + count) & 1, abort)) {
          if (lane == 0) kp_timeout(abort, 0x5a);
          break;
        }
        own0 += count + 1;
        own1 += count;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<1>(tmem_base, KP_TMEM_COLS);
  }
}

// Join the parts of the unit that begins in CTA blockIdx.x's stretch, in CTA
// order: M = max m_p, O = sum 2^(m_p - M) O_p / sum 2^(m_p - M) l_p, with the M so
// far carried along, so that no load waits for a maximum.  A thread takes
// eight columns of KPJ_R rows, the lanes four rows of eight such chunks: whole
// lines of the parts, whose rows stand side by side in 32 bytes, and of O.  (With
// four columns side by side, half sectors of 16 lines a load, the 2048-token
// chunk took 226 us instead of 219; one or four rows a thread: 219, 223.)
constexpr int KPJ_THREADS = 256;
constexpr int KPJ_R = 2;                       // rows of a thread
template <int D>
__global__ void __launch_bounds__(KPJ_THREADS)
kv_prompt_join_kernel(const KpArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const KpJoin* join = a.joins + blockIdx.x;
  const int live = __ldcg(&join->live);
  const int warp = (blockIdx.y * KPJ_THREADS + threadIdx.x) >> 5, lane = threadIdx.x & 31;
  const int r0 = 4 * KPJ_R * (warp / (D / 64)) + (lane & 3);
  const int col = 64 * (warp % (D / 64)) + 8 * (lane >> 2);
  if (r0 >= live) return;
  constexpr long long PART = KP_ROWS * (D + 2);
  const int n = __ldcg(&join->parts);
  const float* first = a.ws + __ldcg(&join->first_slot) * PART;
  const float* rest = a.ws + 2ll * blockIdx.x * PART;
  const int row0 = __ldcg(&join->row0), head = __ldcg(&join->head);
  const long long q0 = __ldcg(&join->q0);
  float top[KPJ_R], sum[KPJ_R], acc[KPJ_R][8];
#pragma unroll
  for (int i = 0; i < KPJ_R; ++i) {
    top[i] = -INFINITY;
    sum[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.0f;
  }
#pragma unroll 2
  for (int p = 0; p < n; ++p) {
    const float* part = p == 0 ? first : rest + 2 * p * PART;
    float mp[KPJ_R], lp[KPJ_R], v[KPJ_R][8];
#pragma unroll
    for (int i = 0; i < KPJ_R; ++i) {
      const int r = min(r0 + 4 * i, live - 1);           // (a row too many is not stored)
      mp[i] = __ldcg(part + KP_ROWS * D + r);
      lp[i] = __ldcg(part + KP_ROWS * (D + 1) + r);
      ld_global_cg_v8(part + (col / 8 * KP_ROWS + r) * 8, v[i]);
    }
#pragma unroll
    for (int i = 0; i < KPJ_R; ++i) {
      const float t = fmaxf(top[i], mp[i]);
      const float before = top[i] == t ? 1.0f : ex2_approx(top[i] - t);
      const float w = mp[i] == t ? 1.0f : ex2_approx(mp[i] - t);
      top[i] = t;
      sum[i] = fmaf(w, lp[i], sum[i] * before);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[i][e] = fmaf(w, v[i][e], acc[i][e] * before);
    }
  }
#pragma unroll
  for (int i = 0; i < KPJ_R; ++i) {
    if (r0 + 4 * i >= live) break;
    const float inv = kv_inverse(sum[i], top[i] != -INFINITY);
    const int row = row0 + r0 + 4 * i, token = row / a.v.group;
    const long long out =
        (q0 + token) * a.o_ts + (head * a.v.group + row - token * a.v.group) * a.o_hs + col;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] *= inv;
    kv_store8(a.O, a.o_dtype, out, acc[i]);
  }
}

template <int FMT, int D>
cudaError_t kp_run(const CUtensorMap& tk, const CUtensorMap& tv, const KpArgs& a, int sms,
                   cudaStream_t st) {
  auto kern = kv_prompt_kernel<FMT, D>;
  using L = KpSmem<D>;
  static std::atomic<bool> attr_set[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !attr_set[dev].load(std::memory_order_relaxed)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALLOC);
    if (e != cudaSuccess) return e;
    // setmaxnreg.inc waits for registers that the launch must have allocated
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * KP_THREADS < KP_REGS_LOW * 128 + KP_REGS_SOFT * 256 + KP_REGS_CONV * 128)
      return cudaErrorInvalidConfiguration;
    if (dev < 64) attr_set[dev].store(true, std::memory_order_relaxed);
  }
  kern<<<sms, KP_THREADS, L::ALLOC, st>>>(tk, tv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || a.ws == nullptr) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms, KP_ROWS * (D / 8) / (KPJ_THREADS * KPJ_R));
  cfg.blockDim = dim3(KPJ_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_prompt_join_kernel<D>, a);
}

}  // namespace

int64_t kv_prompt_max_requests() { return KP_MAX_REQUESTS; }

size_t kv_prompt_workspace_bytes(int64_t d, int sms) {
  return static_cast<size_t>(sms) * (2 * KP_ROWS * (d + 2) * 4 + sizeof(KpJoin)) + 16;
}

cudaError_t launch_kv_prompt(const KvAttn& q, int sms, cudaStream_t st) {
  const KvCache& c = q.cache;
  KpArgs a{};
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
  if (q.ws && q.ws_bytes >= kv_prompt_workspace_bytes(c.d, sms)) {
    // the parts from a 32-byte boundary on
    char* ws = static_cast<char*>(q.ws) + (reinterpret_cast<uintptr_t>(q.ws) & 16);
    a.ws = reinterpret_cast<float*>(ws);
    a.joins = reinterpret_cast<KpJoin*>(ws + static_cast<int64_t>(sms) * 2 * KP_ROWS * (c.d + 2) * 4);
  }
  CUtensorMap tk, tv;
  if (!kv_tensor_map(&tk, c.k, c) || !kv_tensor_map(&tv, c.v, c)) return cudaErrorInvalidValue;
  const bool d64 = c.d == 64;
  switch (c.fmt) {
    case FMT_E4M3:
      return d64 ? kp_run<FMT_E4M3, 64>(tk, tv, a, sms, st) : kp_run<FMT_E4M3, 128>(tk, tv, a, sms, st);
    case FMT_E5M2:
      return d64 ? kp_run<FMT_E5M2, 64>(tk, tv, a, sms, st) : kp_run<FMT_E5M2, 128>(tk, tv, a, sms, st);
    default:
      return d64 ? kp_run<FMT_INT8, 64>(tk, tv, a, sms, st) : kp_run<FMT_INT8, 128>(tk, tv, a, sms, st);
  }
}

unsigned fetch_and_clear_status_kvp(cudaError_t* err) {
  unsigned v = 0, z = 0;
  *err = cudaMemcpyFromSymbol(&v, g_status_kvp, sizeof(v));
  if (*err == cudaSuccess) *err = cudaMemcpyToSymbol(g_status_kvp, &z, sizeof(z));
  return v;
}

}  // namespace mxk
