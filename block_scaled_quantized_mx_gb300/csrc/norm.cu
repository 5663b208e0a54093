// norm.cu -- the residual's addition, the root-mean-square norm and the MX
// quantization of its result in one pass, and an MX tensor's values as a plain
// matrix.
//
//   h = x + r,  r' = round(h),  y_k = h_k / sqrt(mean_k h_k^2 + eps) * w_k,
//   y quantized as quantize.cu would (mx_rule.cuh).
//
// Bound: HBM.  x and r are read once and r', the codes and the scales written
// once: a row's values stay in registers between the sum of squares and the
// conversion, one CTA to a row, 8 consecutive values (16 bytes of 16-bit
// operands) a thread and load, all of a thread's loads on their way together.  A
// block of 32 is four lanes' values, so its maximum takes two shuffles; four
// blocks' scales, one 32-bit word of the row's atom, take two more.  The sum is
// added in a fixed order.
// Measured: 8192 x 8192, bf16 with a bf16 residual, E4M3: 77 us, 6.1 TB/s, 0.90 of the copy
// rate; 4097 x 5120, bf16 with an fp32 residual, E2M1: 37 us, 0.88; 64 x 4096: 2.4 us, a launch
// and two dependent reads.  The values of 8192 x 8192 E4M3 codes as bf16: 32 us, 0.94.
//
// Precision: h, the sum of squares (each thread's, then by halves within a warp, then
// the warps in order) and y are fp32; r' alone is rounded to its type.  Squares that
// overflow (|h| from 2^64 / sqrt(K) on) are summed again, with eps, in units of 2^144; h itself
// is not scaled, so that what is small beside them keeps its bits.  eps is 1e-30 at least, so
// that squares too small for fp32 do not matter beside it.
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "layer_common.cuh"
#include "mx_rule.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

struct NormArgs {
  const void* x;
  const void* r;
  void* r_out;
  const float* w;
  long long x_ld, r_ld, o_ld;
  int x_bf16, r_bf16;
  int chunks;                 // of 8 values, in a row
  int fmt;
  float eps;
  long long rows;
  long long k_atoms;
  uint8_t* data;
  uint8_t* sf;
};

// What a chunk of 8 values of a 16-bit (W = 1) or 32-bit (W = 2) operand takes.
template <int W>
struct Raw8 {
  uint4 v[W == 0 ? 1 : W];
};
template <int W>
__device__ __forceinline__ void load8(Raw8<W>& a, const void* p, long long at) {
  if constexpr (W == 1) {
    a.v[0] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  } else if constexpr (W == 2) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + at);
    a.v[0] = q[0];
    a.v[1] = q[1];
  }
}
template <int W>
__device__ __forceinline__ void values8(const Raw8<W>& a, int bf16, float (&x)[8]) {
  if constexpr (W == 1) {
    const uint32_t w[4] = {a.v[0].x, a.v[0].y, a.v[0].z, a.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack16x2(w[i], bf16, x[2 * i], x[2 * i + 1]);
  } else if constexpr (W == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = __uint_as_float(a.v[i].x);
      x[4 * i + 1] = __uint_as_float(a.v[i].y);
      x[4 * i + 2] = __uint_as_float(a.v[i].z);
      x[4 * i + 3] = __uint_as_float(a.v[i].w);
    }
  }
}

// Sum over the CTA's threads, the same in each of them.  `sm`: a float per warp.
__device__ __forceinline__ float row_sum(float v, float* sm) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  const int warps = blockDim.x >> 5;
  float s = sm[0];
  for (int i = 1; i < warps; ++i) s += sm[i];
  return s;
}

template <int FMT>
__device__ __forceinline__ void store_codes(uint8_t* data, long long at, const float (&y)[8],
                                            float inv) {
  const uint32_t a = codes4<FMT>(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
  const uint32_t b = codes4<FMT>(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv);
  if (FMT == FMT_E2M1)
    *reinterpret_cast<uint32_t*>(data + at / 2) = a | (b << 16);
  else
    *reinterpret_cast<uint2*>(data + at) = make_uint2(a, b);
}

// The largest of a, |b| and |c|, a NaN if one of them is.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// XW, RW: what a chunk of x and of r takes (RW 0: there is no r); CH: chunks a
// thread.
template <int XW, int RW, int CH>
__global__ void __launch_bounds__(CH <= 2 ? 1024 : 512) rmsnorm_quantize_kernel(const NormArgs a) {
  __shared__ float sm_sum[64];
  const long long row = blockIdx.x;
  const int lane = threadIdx.x & 31;
  wait_for_stream();
  if (row >= a.rows) {                       // rows that pad the last atom: scales 0
    for (int c = 16 * threadIdx.x; c < a.chunks; c += 16 * blockDim.x)
      *reinterpret_cast<uint32_t*>(a.sf + sf_offset(row, c / 4, a.k_atoms)) = 0u;
    return;
  }
  Raw8<XW> rx[CH];
  Raw8<RW> rr[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    if (c < a.chunks) {
      load8<XW>(rx[i], a.x, row * a.x_ld + 8ll * c);
      if constexpr (RW > 0) load8<RW>(rr[i], a.r, row * a.r_ld + 8ll * c);
    }
  }
  float h[CH][8], sum = 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
#pragma unroll
    for (int e = 0; e < 8; ++e) h[i][e] = 0.0f;
    if (c < a.chunks) {
      values8<XW>(rx[i], a.x_bf16, h[i]);
      if constexpr (RW > 0) {
        float r[8];
        values8<RW>(rr[i], a.r_bf16, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += r[e];
        const long long at = row * a.o_ld + 8ll * c;
        if constexpr (RW == 2) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.r_out) + at);
          o[0] = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
          o[1] = make_float4(h[i][4], h[i][5], h[i][6], h[i][7]);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = a.r_bf16 ? cvt_bf16x2(h[i][2 * e], h[i][2 * e + 1])
                            : cvt_f16x2(h[i][2 * e], h[i][2 * e + 1]);
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.r_out) + at) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
    }
  }
  const float K = 8.0f * static_cast<float>(a.chunks);
  sum = row_sum(sum, sm_sum);
  float f = __frsqrt_rn(sum / K + a.eps);
  if (!(sum <= 3.402823466e38f)) {           // the whole CTA
    constexpr float unit = 2.1175824e-22f;   // 2^-72
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e] * unit, h[i][e] * unit, sum);
    // (2^-128 at least, where a subnormal still has 21 bits; 0 beside an infinity)
    f = __frsqrt_rn(row_sum(sum, sm_sum + 32) / K + a.eps * unit * unit) * unit;
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    float y[8];
    // y of the chunk, and the largest |y| of its block.  FAR: not by way of an h f below the
    // normal numbers, from where a weight may bring the product back.
    auto normed = [&](auto far, float& heaviest) {
      constexpr bool FAR = decltype(far)::value;
      float most = 0.0f;
      heaviest = 0.0f;
      if (c < a.chunks) {
        const float4* w = reinterpret_cast<const float4*>(a.w) + 2 * c;
        const float4 w0 = w[0], w1 = w[1];
        const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = h[i][e] * f;
          y[e] = n * ww[e];
          if (FAR && fabsf(n) < 1.17549435e-38f && h[i][e] != 0.0f) {
            const float by = f * ww[e];      // (beyond fp32 for a subnormal h under 2^105 and more)
            if (fabsf(by) <= 3.402823466e38f) y[e] = h[i][e] * by;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          most = max3_abs(most, y[e], y[e + 1]);
          if (!FAR) heaviest = max3_abs(heaviest, ww[e], ww[e + 1]);
        }
      }
      uint32_t top = __float_as_uint(most);
      top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
      return max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    };
    // Such an h f is off by 2^-150, y by 2^-90 under a weight of 2^60: 2^-27 of the smallest step
    // of a code in a block whose largest y is 2^-32.
    float heaviest;
    uint32_t top = normed(std::false_type{}, heaviest);
    if (__any_sync(0xFFFFFFFFu, c < a.chunks && (top < 0x2F800000u || !(heaviest < 1.1529215e18f))))
      top = normed(std::true_type{}, heaviest);
    uint32_t code;
    float inv;
    block_scale(top, emax_of_fmt(a.fmt), code, inv);
    if (c < a.chunks) {
      const long long at = row * 8ll * a.chunks + 8ll * c;
      if (a.fmt == FMT_E4M3)
        store_codes<FMT_E4M3>(a.data, at, y, inv);
      else if (a.fmt == FMT_E5M2)
        store_codes<FMT_E5M2>(a.data, at, y, inv);
      else
        store_codes<FMT_E2M1>(a.data, at, y, inv);
    }
    // 16 lanes hold four blocks: one word of the atom's row (0 for blocks behind K)
    uint32_t word = c < a.chunks ? code << (8 * ((lane >> 2) & 3)) : 0u;
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 4);
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 8);
    if ((lane & 15) == 0 && c < a.chunks)
      *reinterpret_cast<uint32_t*>(a.sf + sf_offset(row, c / 4, a.k_atoms)) = word;
  }
}

template <int XW, int RW>
cudaError_t norm_run(const NormArgs& a, unsigned ctas, int ch, int threads, cudaStream_t st) {
  switch (ch) {
    case 1: return launch_early(rmsnorm_quantize_kernel<XW, RW, 1>, ctas, threads, 0, 1, st, a);
    case 2: return launch_early(rmsnorm_quantize_kernel<XW, RW, 2>, ctas, threads, 0, 1, st, a);
    case 4: return launch_early(rmsnorm_quantize_kernel<XW, RW, 4>, ctas, threads, 0, 1, st, a);
    default: return launch_early(rmsnorm_quantize_kernel<XW, RW, 8>, ctas, threads, 0, 1, st, a);
  }
}

// ------------------------------------------------------------------ values

struct DequantArgs {
  const uint8_t* data;
  const uint8_t* sf;
  void* out;
  long long ld, units, k_atoms;   // units: of 16 values, in the whole matrix
  uint32_t per_row;
  int dtype;
};

// Four codes, element 0 in the lowest bits, as values.
template <int FMT>
__device__ __forceinline__ void code_values4(uint32_t w, float (&x)[4]) {
  if constexpr (FMT == FMT_E4M3 || FMT == FMT_E5M2) {
    f16x2_to_f32(FMT == FMT_E4M3 ? cvt_f16x2_e4m3x2(w & 0xFFFFu) : cvt_f16x2_e5m2x2(w & 0xFFFFu), x[0], x[1]);
    f16x2_to_f32(FMT == FMT_E4M3 ? cvt_f16x2_e4m3x2(w >> 16) : cvt_f16x2_e5m2x2(w >> 16), x[2], x[3]);
  } else if constexpr (FMT == FMT_E2M1) {
    f16x2_to_f32(cvt_f16x2_e2m1x2(w & 0xFFu), x[0], x[1]);
    f16x2_to_f32(cvt_f16x2_e2m1x2((w >> 8) & 0xFFu), x[2], x[3]);
  } else {
    constexpr int BITS = FMT == FMT_INT8 ? 8 : FMT == FMT_INT4 ? 4 : 2;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = static_cast<float>(static_cast<int32_t>(w << (32 - BITS * (i + 1))) >> (32 - BITS));
  }
}

// A thread takes units of 16 values, DQ_BATCH of them with their loads together.
constexpr int DQ_THREADS = 256, DQ_BATCH = 4;
template <int FMT>
__global__ void __launch_bounds__(DQ_THREADS) dequantize_kernel(const DequantArgs a) {
  constexpr int BITS = FMT == FMT_INT2 ? 2 : (FMT == FMT_E2M1 || FMT == FMT_INT4) ? 4 : 8;
  const long long u0 = static_cast<long long>(blockIdx.x) * (DQ_THREADS * DQ_BATCH) + threadIdx.x;
  wait_for_stream();
  uint32_t w[DQ_BATCH][4];
  uint32_t scale[DQ_BATCH];
  long long row[DQ_BATCH];
  uint32_t col[DQ_BATCH];
#pragma unroll
  for (int i = 0; i < DQ_BATCH; ++i) {
    const long long u = u0 + i * DQ_THREADS;
    if (u >= a.units) break;
    row[i] = (u >> 32) == 0 ? static_cast<uint32_t>(u) / a.per_row : u / a.per_row;
    col[i] = static_cast<uint32_t>(u - row[i] * a.per_row);
    if constexpr (BITS == 8) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4*>(a.data) + u);
      w[i][0] = v.x;
      w[i][1] = v.y;
      w[i][2] = v.z;
      w[i][3] = v.w;
    } else if constexpr (BITS == 4) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(a.data) + u);
      w[i][0] = v.x;
      w[i][1] = v.x >> 16;
      w[i][2] = v.y;
      w[i][3] = v.y >> 16;
    } else {
      const uint32_t v = __ldcs(reinterpret_cast<const uint32_t*>(a.data) + u);
#pragma unroll
      for (int q = 0; q < 4; ++q) w[i][q] = v >> (8 * q);
    }
    scale[i] = a.sf[sf_offset(row[i], col[i] / 2, a.k_atoms)];
  }
#pragma unroll
  for (int i = 0; i < DQ_BATCH; ++i) {
    if (u0 + i * DQ_THREADS >= a.units) break;
    const float f = ue8m0_value(scale[i]);
    float x[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4];
      code_values4<FMT>(w[i][q], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * q + e] = v[e] * f;
    }
    const long long at = row[i] * a.ld + 16ll * col[i];
    if (a.dtype == DT_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
    } else {
      uint32_t p[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        p[q] = a.dtype == DT_BF16 ? cvt_bf16x2(x[2 * q], x[2 * q + 1]) : cvt_f16x2(x[2 * q], x[2 * q + 1]);
      uint16_t* o = static_cast<uint16_t*>(a.out) + at;
      if ((reinterpret_cast<uintptr_t>(o) & 31) == 0) {
        st_global_v8(o, p);
      } else {
        reinterpret_cast<uint4*>(o)[0] = make_uint4(p[0], p[1], p[2], p[3]);
        reinterpret_cast<uint4*>(o)[1] = make_uint4(p[4], p[5], p[6], p[7]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rmsnorm_quantize(const void* x, int x_dtype, int64_t x_ld, const void* r,
                                    int r_dtype, int64_t r_ld, const float* w, float eps,
                                    void* r_out, int64_t o_ld, int fmt, int64_t rows, int64_t K,
                                    void* data, uint8_t* sf, cudaStream_t st) {
  NormArgs a{};
  a.x = x;
  a.r = r;
  a.r_out = r_out;
  a.w = w;
  a.x_ld = x_ld;
  a.r_ld = r_ld;
  a.o_ld = o_ld;
  a.x_bf16 = x_dtype == DT_BF16;
  a.r_bf16 = r_dtype == DT_BF16;
  a.chunks = static_cast<int>(K / 8);
  a.fmt = fmt;
  a.eps = eps;
  a.rows = rows;
  a.k_atoms = sf_k_atoms(K);
  a.data = static_cast<uint8_t*>(data);
  a.sf = sf;
  const unsigned ctas = static_cast<unsigned>(sf_row_atoms(rows) * SF_ATOM_ROWS);
  // As few chunks a thread as 1024 threads allow where the rows do not fill the
  // SMs (a row's time is what counts); where they do, one to 2048 values, two below
  // 8192, four to 16384, so that longer rows have 130 to 512 threads (8192 rows of
  // 8192 with 1, 2, 4 and 8 chunks 104, 95, 77 and 96 us; 4097 of 5120, fp32 residual,
  // 39, 38, 41 and 50; where two and four cross between those widths is not measured).
  const bool few = rows <= 2 * 152;
  int ch = a.chunks <= 256 ? 1 : a.chunks < 1024 ? 2 : a.chunks <= 2048 ? 4 : 8;
  if (few && a.chunks <= 2048) ch = a.chunks <= 1024 ? 1 : 2;
  const int threads = ((a.chunks + ch - 1) / ch + 31) / 32 * 32;
  const int rw = r == nullptr ? 0 : r_dtype == DT_F32 ? 2 : 1;
  if (x_dtype == DT_F32)
    return rw == 0 ? norm_run<2, 0>(a, ctas, ch, threads, st)
           : rw == 1 ? norm_run<2, 1>(a, ctas, ch, threads, st) : norm_run<2, 2>(a, ctas, ch, threads, st);
  return rw == 0 ? norm_run<1, 0>(a, ctas, ch, threads, st)
         : rw == 1 ? norm_run<1, 1>(a, ctas, ch, threads, st) : norm_run<1, 2>(a, ctas, ch, threads, st);
}

cudaError_t launch_dequantize(int fmt, const void* data, const uint8_t* sf, int64_t outer, int64_t K,
                              void* out, int dtype, int64_t ld, cudaStream_t st) {
  DequantArgs a{};
  a.data = static_cast<const uint8_t*>(data);
  a.sf = sf;
  a.out = out;
  a.ld = ld;
  a.per_row = static_cast<uint32_t>(K / 16);
  a.units = outer * (K / 16);
  a.k_atoms = sf_k_atoms(K);
  a.dtype = dtype;
  const long long ctas = (a.units + DQ_THREADS * DQ_BATCH - 1) / (DQ_THREADS * DQ_BATCH);
  if (ctas > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(ctas);
  switch (fmt) {
    case FMT_E4M3: return launch_early(dequantize_kernel<FMT_E4M3>, grid, DQ_THREADS, 0, 1, st, a);
    case FMT_E5M2: return launch_early(dequantize_kernel<FMT_E5M2>, grid, DQ_THREADS, 0, 1, st, a);
    case FMT_E2M1: return launch_early(dequantize_kernel<FMT_E2M1>, grid, DQ_THREADS, 0, 1, st, a);
    case FMT_INT8: return launch_early(dequantize_kernel<FMT_INT8>, grid, DQ_THREADS, 0, 1, st, a);
    case FMT_INT4: return launch_early(dequantize_kernel<FMT_INT4>, grid, DQ_THREADS, 0, 1, st, a);
    default: return launch_early(dequantize_kernel<FMT_INT2>, grid, DQ_THREADS, 0, 1, st, a);
  }
}

}  // namespace mxk
