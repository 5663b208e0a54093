// kv_kernel.cuh -- device helpers shared by the attention kernels over the
// 8-bit paged cache: what a request's rows may see, codes to f16, factors.
#pragma once
#include <cstdint>

#include "common.cuh"
#include "gemm_common.cuh"
#include "kv_common.cuh"
#include "ptx.cuh"

namespace mxk {

// What the kernels need of a cache, its tables and its requests.
struct KvView {
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int* table;
  long long table_stride;
  const int* lens;
  const int* cu;
  long long tokens;            // rows of Q
  long long pages;
  int heads;                   // cache heads
  int group;                   // query heads per cache head
  int page_shift;
  int requests;
  int capacity;                // tokens a table row holds
  int causal;
  int window;                  // 0: none
};

inline KvView kv_view(const KvAttn& q) {
  KvView v{};
  v.k_scales = q.cache.k_scales;
  v.v_scales = q.cache.v_scales;
  v.table = q.table;
  v.table_stride = q.table_stride;
  v.lens = q.lens;
  v.cu = q.cu;
  v.tokens = q.tokens;
  v.pages = q.cache.pages;
  v.heads = static_cast<int>(q.cache.heads);
  v.group = static_cast<int>(q.q_heads / q.cache.heads);
  v.page_shift = kv_page_shift(q.cache.page);
  v.requests = static_cast<int>(q.requests);
  const int64_t most = q.width << v.page_shift;
  v.capacity = static_cast<int>(most < 0x7FFFFF00 ? most : 0x7FFFFF00);
  v.causal = q.causal;
  v.window = static_cast<int>(q.window < 0x7FFFFF00 ? q.window : 0x7FFFFF00);
  return v;
}

// One request: its rows of Q (first, count) and its length.  Whatever the
// arrays hold, the rows lie in Q and the length in the table.
struct KvReq {
  long long q0;
  int n;
  int len;
};

__device__ __forceinline__ KvReq kv_request(const KvView& v, int b) {
  KvReq r;
  long long s = v.cu[b], e = v.cu[b + 1];
  s = s < 0 ? 0 : (s > v.tokens ? v.tokens : s);
  e = e < s ? s : (e > v.tokens ? v.tokens : e);
  r.q0 = s;
  r.n = static_cast<int>(e - s);
  const int len = v.lens[b];
  r.len = len < 0 ? 0 : (len > v.capacity ? v.capacity : len);
  return r;
}

// Token i of a request stands at position len - n + i and sees keys
// [first, end): all before its own and itself (causal), or all; with a
// window only the last `window` up to its own position.
__device__ __forceinline__ int kv_first_key(const KvView& v, const KvReq& r, int i) {
  if (v.window <= 0) return 0;
  const long long p = static_cast<long long>(r.len) - r.n + i + 1 - v.window;
  return p > 0 ? static_cast<int>(p) : 0;
}
__device__ __forceinline__ int kv_end_key(const KvView& v, const KvReq& r, int i) {
  if (!v.causal) return r.len;
  const int p = r.len - r.n + i + 1;
  return p > 0 ? p : 0;
}

// The list of all requests' row tiles (`rows` rows each), and the request of a
// tile in it.  Starts are kept in 32 bits.  Rows of Q that belong to one request
// each make `most` tiles at most, a last one that is not full for every request
// included; offsets that go up and down may name rows again and again, in any
// number: the list then ends at `most`, and so do the starts.
struct KvTileList {
  long long most;
  __host__ __device__ KvTileList(long long tokens, int group, int rows, int requests)
      : most((tokens * group + rows - 1) / rows + requests) {}
  __host__ __device__ long long clip(long long at) const { return at < most ? at : most; }
  __host__ __device__ int start(long long at) const { return static_cast<int>(clip(at)); }
  // the last of the requests that begins at or before tile f < clip(their sum)
  static __host__ __device__ int request(const int* starts, int requests, long long f) {
    int lo = 0, hi = requests - 1;
    while (lo < hi) {
      const int m = (lo + hi + 1) >> 1;
      if (starts[m] <= f) lo = m; else hi = m - 1;
    }
    return lo;
  }
};

// Whether the table entry of key j's page is followed: the page begins in front of
// the request's end and does not end in front of `first`, the first key that any
// row sees.  (A page behind the window may belong to another request by now,
// whatever the table still says.)
__device__ __forceinline__ bool kv_follows(const KvView& v, const KvReq& r, int first, int j) {
  return j < r.len && ((j >> v.page_shift) + 1) << v.page_shift > first;
}

// A scale code as a factor: 2^(c - 127); 0xFF is NaN.
__device__ __forceinline__ float kv_scale_value(uint32_t c) {
  return __uint_as_float(c == 0 ? 0x00400000u : c == 0xFFu ? 0x7FC00000u : (c << 23));
}

// A row's running maximum before its first score above -infinity.  Finite, so that
// x_j - m stays -infinity for scores of -infinity, hidden or real: they weigh
// nothing, whatever comes beside them.  A part states it for a row that saw such
// scores only, and -infinity for a row that saw none: where no part has another
// maximum, the first is 0 / 0 and the second 0.
constexpr float KV_NO_MAX = -3.402823466e38f;

// 1 / (the sum of a row's weights): 0 for a row that saw no key, NaN for one
// whose every score was -infinity.
__device__ __forceinline__ float kv_inverse(float sum, bool saw_keys) {
  return sum != 0.0f ? 1.0f / sum : saw_keys ? __uint_as_float(0x7FC00000u) : 0.0f;
}

// The exponents of P.  A row's weights are 2^(x_j - m), and V's pages have scales
// 2^(e_j - 127) of any size, so that neither the largest weight nor the largest
// scale says which products matter.  P is rounded to f16 as
//   2^(x_j - m + e_j - v + 7),
// where v is at least the largest x_j - m + e_j of the keys that the row itself
// sees, less KV_LAZY, and at most that rounded up: the product that weighs most
// stands between 2^6 and 2^15.  Keys that a row does not see, and pages of large
// values that it gives no weight, leave the others' precision alone.  The sum of
// the weights takes 2^(e_j - v + 7) out again.  (m is a score, not one rounded to a
// whole number: the key that it comes from, often most of the row's weight, then
// has no rounding at all.  With m rounded up, outputs in f16 were off by 2.9e-4
// instead of 2.4e-4.)
constexpr float KV_LAZY = 8.0f;            // slack of m and of v
constexpr int KV_P_EXP = 7;
constexpr float KV_NO_V = -300.0f;         // v of a row that has seen nothing: below every other

// m for a row whose next scores are x_top at most.
__device__ __forceinline__ float kv_next_m(float m, float x_top) {
  return x_top > m + KV_LAZY ? x_top : m;
}
// v for a row whose m moved by dm = m_old - m_new, to the next keys' largest
// x_j - m_new + e_j.
__device__ __forceinline__ float kv_next_v(float v, float dm, float top) {
  const float r = fmaxf(v + dm, KV_NO_V);
  return top > r + KV_LAZY ? ceilf(top) : r;
}

// What O, in units of 2^v_old at m_old, is multiplied by when they become v and m.
__device__ __forceinline__ float kv_move_o(float m_old, float m_new, float v_old, float v_new) {
  return ex2_approx((m_old - m_new) + (v_old - v_new));
}

// e_j - v + 7 of a page.  Below 2^-60 P is 0 in f16 whatever it is exactly, and
// the sum still gets the weight.
__device__ __forceinline__ float kv_p_shift(float e, float v) {
  return fmaxf(e - v + static_cast<float>(KV_P_EXP), -60.0f);
}

// 2^-b of such a shift (0 beyond 126: weights of less than 2^-110).
__device__ __forceinline__ float kv_unshift(float b) { return ex2_approx(-b); }

// The unit of O, 2^(v - 127 - 7), as two factors: v goes from -16 to 262.
__device__ __forceinline__ void kv_o_unit(float v, float& f0, float& f1) {
  const float e = v - static_cast<float>(127 + KV_P_EXP), half = floorf(0.5f * e);
  f0 = ex2_approx(half);
  f1 = ex2_approx(e - half);
}

// For a row whose largest |value| has the bit pattern `top`: powers of two
// that bring it into [1, 2) and back.  Rows of zeros, infinities and NaN
// stay as they are.
__device__ __forceinline__ void kv_row_factors(uint32_t top, float& down, float& up) {
  const uint32_t e = top >> 23;
  if (e == 0 || e == 255) {
    down = up = 1.0f;
    return;
  }
  const uint32_t c = e < 2 ? 2 : (e > 252 ? 252 : e);
  down = __uint_as_float((254 - c) << 23);
  up = __uint_as_float(c << 23);
}

// Four codes -> two f16 pairs, exactly.
template <int FMT>
__device__ __forceinline__ void kv_f16_pairs(uint32_t w, uint32_t& p0, uint32_t& p1) {
  if constexpr (FMT == FMT_E4M3) {
    p0 = cvt_f16x2_e4m3x2(w & 0xFFFFu);
    p1 = cvt_f16x2_e4m3x2(w >> 16);
  } else if constexpr (FMT == FMT_E5M2) {
    // an E5M2 code is the high byte of the f16 of the same value
    p0 = __byte_perm(w, 0u, 0x1404);
    p1 = __byte_perm(w, 0u, 0x3424);
  } else {
    // q + 128 under the byte 0x64 is the f16 1024 + (q + 128)
    const uint32_t u = w ^ 0x80808080u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p0) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p1) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
  }
}

__device__ __forceinline__ uint2 kv_ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void kv_bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Four consecutive outputs at element `at`.
__device__ __forceinline__ void kv_store4(void* O, int o_dtype, long long at, float4 v) {
  if (o_dtype == DT_F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(O) + at) = v;
  } else if (o_dtype == DT_BF16) {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(O) + at) =
        make_uint2(cvt_bf16x2(v.x, v.y), cvt_bf16x2(v.z, v.w));
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(O) + at) =
        make_uint2(cvt_f16x2(v.x, v.y), cvt_f16x2(v.z, v.w));
  }
}

// Eight consecutive outputs at element `at`.
__device__ __forceinline__ void kv_store8(void* O, int o_dtype, long long at, const float (&v)[8]) {
  if (o_dtype == DT_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(O) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    const bool bf = o_dtype == DT_BF16;
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(O) + at) =
        make_uint4(bf ? cvt_bf16x2(v[0], v[1]) : cvt_f16x2(v[0], v[1]),
                   bf ? cvt_bf16x2(v[2], v[3]) : cvt_f16x2(v[2], v[3]),
                   bf ? cvt_bf16x2(v[4], v[5]) : cvt_f16x2(v[4], v[5]),
                   bf ? cvt_bf16x2(v[6], v[7]) : cvt_f16x2(v[6], v[7]));
  }
}

// One box of the K or V plane: the P x d codes of a page of one head, rows
// swizzled over 128 bytes (d 128) or 64 (d 64).
inline bool kv_tensor_map(CUtensorMap* m, const void* p, const KvCache& c) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(c.d),
                        static_cast<cuuint64_t>(c.pages * c.heads * c.page)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(c.d)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(c.d), static_cast<cuuint32_t>(c.page)};
  cuuint32_t estr[2] = {1, 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, p, dims, strides, box, estr,
                      c.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

}  // namespace mxk
