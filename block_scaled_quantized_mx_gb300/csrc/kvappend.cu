// kvappend.cu -- new keys and values into the 8-bit paged cache.
//
// A page of one head has one power-of-two scale.  For the tokens that a call
// adds to it, e is the OCP MX scale code of their largest magnitude (the rule
// of mx_rule.cuh over the block); a page whose first token this call writes
// gets s = e, one that held tokens before gets s = max(s_old, e), and where
// the scale grew the codes before them are rounded again, to nearest, as
// code * 2^(s_old - s).  New codes are round_sat(x * 2^(127 - s)).  A NaN or an
// infinity makes the page's scale 0xFF (NaN), its new codes 0, and it stays
// NaN until the page is begun anew.
//
// Bound: HBM, 2 bytes read and 1 written per value.  One CTA of 128 threads
// per (run of tokens in one page, head, K or V): the run's values (at most
// 128 x 128) are read once, 16 bytes a load, all loads in flight together, and
// stay packed in registers between the maximum and the conversion.  A run is
// found from the slots: it begins at a token whose predecessor's slot is not
// the one before, or whose slot is a page's first.  A CTA looks for beginnings
// among `seg` tokens: as many as a page has, so that a prompt gives a CTA one
// run, and fewer when that leaves SMs idle (single-token steps: each token
// begins a run).
// Measured: 32 prompts of 512 tokens, 8 heads of 128, pages of 64: 18.0 us, 5.6
// TB/s, 0.82 of the copy rate (at 96 registers, five CTAs an SM instead of
// eight, 20.5 us); 64 single tokens: 4.1 us, the launch and three dependent
// reads.
#include <cstdint>

#include "common.cuh"
#include "kv_common.cuh"
#include "mx_rule.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int AP_THREADS = 128;

struct AppendArgs {
  const uint16_t *k, *v;
  long long k_ts, k_hs, v_ts, v_hs;
  uint8_t *k_codes, *v_codes;
  uint8_t *k_scales, *v_scales;
  const long long* slots;
  long long tokens;
  long long pages;
  int heads;
  int d_shift;                // log2 of d
  int page_shift;
  int seg_shift;
  int bf16;
};

__device__ __forceinline__ void unpack16(uint32_t w, int bf16, float& lo, float& hi) {
  if (bf16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  } else {
    f16x2_to_f32(w, lo, hi);
  }
}

// One 32-bit word of four codes times f (a power of two), rounded again.
template <int FMT>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  float x[4];
  if (FMT == FMT_INT8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = static_cast<float>(static_cast<int8_t>(w >> (8 * i)));
  } else {
    const uint32_t h0 = FMT == FMT_E5M2 ? cvt_f16x2_e5m2x2(w & 0xFFFFu) : cvt_f16x2_e4m3x2(w & 0xFFFFu);
    const uint32_t h1 = FMT == FMT_E5M2 ? cvt_f16x2_e5m2x2(w >> 16) : cvt_f16x2_e4m3x2(w >> 16);
    f16x2_to_f32(h0, x[0], x[1]);
    f16x2_to_f32(h1, x[2], x[3]);
  }
  return codes4<FMT>(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}

// NP: 16-byte loads per thread that cover a whole page of one head.
template <int FMT, int NP>
__global__ void __launch_bounds__(AP_THREADS, NP == 16 ? 4 : 8) kv_append_kernel(const AppendArgs a) {
  __shared__ uint32_t sm_max[AP_THREADS / 32];
  __shared__ int sm_len;
  __shared__ uint32_t sm_begin[4];          // one bit per token of the segment
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int head = blockIdx.y;
  const bool is_k = blockIdx.z == 0;
  const int P = 1 << a.page_shift, seg = 1 << a.seg_shift;
  const long long t0 = static_cast<long long>(blockIdx.x) << a.seg_shift;
  {
    const long long t = t0 + tid;
    bool begins = false;
    if (tid < seg && t < a.tokens) {
      const long long s = a.slots[t];
      begins = s >= 0 && (s >> a.page_shift) < a.pages &&
               ((s & (P - 1)) == 0 || t == 0 || a.slots[t - 1] != s - 1);
    }
    const uint32_t bits = __ballot_sync(0xFFFFFFFFu, begins);
    if (lane == 0) sm_begin[warp] = bits;
  }
  __syncthreads();
  const uint16_t* src = (is_k ? a.k : a.v) + static_cast<long long>(head) * (is_k ? a.k_hs : a.v_hs);
  const long long ts = is_k ? a.k_ts : a.v_ts;
  const int row_shift = a.d_shift - 3;      // 16-byte chunks (8 values) per row: 2^row_shift
  for (int word = 0; word < 4; ++word) {
    uint32_t bits = sm_begin[word];
    while (bits) {
      const long long t = t0 + 32 * word + (__ffs(bits) - 1);
      bits &= bits - 1;
      const long long slot = a.slots[t];
      const int off = static_cast<int>(slot & (P - 1));
      // the run's length: up to the page's end, as long as slots go on by one
      const int most = static_cast<int>(min(static_cast<long long>(P - off), a.tokens - t));
      if (tid == 0) sm_len = most;
      __syncthreads();
      if (tid < most && a.slots[t + tid] != slot + tid) atomicMin(&sm_len, tid);
      __syncthreads();
      const int n = sm_len;
      const long long unit = (slot >> a.page_shift) * a.heads + head;
      uint8_t* scale_at = (is_k ? a.k_scales : a.v_scales) + unit;
      uint4 buf[NP];
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int c = i * AP_THREADS + tid, r = c >> row_shift;
        buf[i] = make_uint4(0, 0, 0, 0);
        if (r < n)
          buf[i] = *reinterpret_cast<const uint4*>(src + (t + r) * ts +
                                                   ((c & ((1 << row_shift) - 1)) << 3));
      }
      const uint32_t s_old = off ? *scale_at : 0u;
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint32_t w[4] = {buf[i].x, buf[i].y, buf[i].z, buf[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float lo, hi;
          unpack16(w[e], a.bf16, lo, hi);
          amax = max(amax, max(abs_bits(lo), abs_bits(hi)));
        }
      }
      amax = __reduce_max_sync(0xFFFFFFFFu, amax);
      if (lane == 0) sm_max[warp] = amax;
      __syncthreads();                      // also: every thread has read the old scale
      amax = max(max(sm_max[0], sm_max[1]), max(sm_max[2], sm_max[3]));
      uint32_t s;
      float inv;
      block_scale(amax, emax_of<FMT>(), s, inv);
      if (s_old > s) s = s_old;
      // 2^(127 - s): the subnormal 2^-127 for s = 254; nothing for a NaN scale
      inv = s == 0xFFu ? 0.0f : __uint_as_float(s == 254u ? 0x00400000u : (254u - s) << 23);
      uint8_t* page = (is_k ? a.k_codes : a.v_codes) + ((unit << a.page_shift) << a.d_shift);
      if (off && s > s_old && s != 0xFFu) {
        // the codes before the run, under the new scale
        const int shift = static_cast<int>(s - s_old);
        const float f = shift > 126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(127 - shift) << 23);
        const int chunks = off << (a.d_shift - 4);
        for (int c = tid; c < chunks; c += AP_THREADS) {
          uint4* p = reinterpret_cast<uint4*>(page) + c;
          uint4 w = *p;
          w.x = rescale4<FMT>(w.x, f);
          w.y = rescale4<FMT>(w.y, f);
          w.z = rescale4<FMT>(w.z, f);
          w.w = rescale4<FMT>(w.w, f);
          *p = w;
        }
      }
      if (tid == 0) *scale_at = static_cast<uint8_t>(s);
      uint8_t* dst = page + (static_cast<long long>(off) << a.d_shift);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const int c = i * AP_THREADS + tid, r = c >> row_shift;
        if (r < n) {
          const uint32_t w[4] = {buf[i].x, buf[i].y, buf[i].z, buf[i].w};
          float x[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            unpack16(w[e], a.bf16, x[2 * e], x[2 * e + 1]);
            x[2 * e] *= inv;
            x[2 * e + 1] *= inv;
          }
          uint2 o = make_uint2(codes4<FMT>(x[0], x[1], x[2], x[3]),
                               codes4<FMT>(x[4], x[5], x[6], x[7]));
          if (s == 0xFFu) o = make_uint2(0u, 0u);   // 0 * infinity is a NaN code
          *reinterpret_cast<uint2*>(dst + 8 * static_cast<long long>(c)) = o;
        }
      }
      __syncthreads();                      // sm_len and sm_max are free again
    }
  }
}

template <int FMT>
cudaError_t append_run(const AppendArgs& a, int np, dim3 grid, cudaStream_t st) {
  switch (np) {
    case 1: kv_append_kernel<FMT, 1><<<grid, AP_THREADS, 0, st>>>(a); break;
    case 2: kv_append_kernel<FMT, 2><<<grid, AP_THREADS, 0, st>>>(a); break;
    case 4: kv_append_kernel<FMT, 4><<<grid, AP_THREADS, 0, st>>>(a); break;
    case 8: kv_append_kernel<FMT, 8><<<grid, AP_THREADS, 0, st>>>(a); break;
    default: kv_append_kernel<FMT, 16><<<grid, AP_THREADS, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_append(const KvCache& c, const void* K, const void* V, int dtype,
                             int64_t tokens, int64_t k_ts, int64_t k_hs, int64_t v_ts,
                             int64_t v_hs, const int64_t* slots, cudaStream_t st) {
  AppendArgs a{};
  a.k = static_cast<const uint16_t*>(K);
  a.v = static_cast<const uint16_t*>(V);
  a.k_ts = k_ts;
  a.k_hs = k_hs;
  a.v_ts = v_ts;
  a.v_hs = v_hs;
  a.k_codes = c.k;
  a.v_codes = c.v;
  a.k_scales = c.k_scales;
  a.v_scales = c.v_scales;
  a.slots = reinterpret_cast<const long long*>(slots);
  a.tokens = tokens;
  a.pages = c.pages;
  a.heads = static_cast<int>(c.heads);
  a.d_shift = c.d == 64 ? 6 : 7;
  a.page_shift = kv_page_shift(c.page);
  a.bf16 = dtype == DT_BF16;
  // segments of up to a page's tokens, shortened until there are about 16
  // CTAs for each of the 152 SMs
  a.seg_shift = a.page_shift;
  while (a.seg_shift > 0 && ((tokens + (1ll << a.seg_shift) - 1) >> a.seg_shift) * c.heads * 2 < 2432)
    --a.seg_shift;
  const int64_t segs = (tokens + (1ll << a.seg_shift) - 1) >> a.seg_shift;
  const dim3 grid(static_cast<unsigned>(segs), static_cast<unsigned>(c.heads), 2);
  const int np = static_cast<int>(c.page * c.d / 8 / AP_THREADS);
  switch (c.fmt) {
    case FMT_E4M3: return append_run<FMT_E4M3>(a, np, grid, st);
    case FMT_E5M2: return append_run<FMT_E5M2>(a, np, grid, st);
    default: return append_run<FMT_INT8>(a, np, grid, st);
  }
}

}  // namespace mxk
