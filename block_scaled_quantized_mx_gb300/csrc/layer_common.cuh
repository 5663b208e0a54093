// layer_common.cuh -- what stands around the products and the attention of a
// decoder layer: norm.cu, rope.cu.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mxk {

// The two values of a word of 16-bit elements.
__device__ __forceinline__ void unpack16x2(uint32_t w, int bf16, float& lo, float& hi) {
  if (bf16) {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xFFFF0000u);
  } else {
    f16x2_to_f32(w, lo, hi);
  }
}

// A scale code as a factor: 2^(c - 127); 0xFF is NaN.
__device__ __forceinline__ float ue8m0_value(uint32_t c) {
  return __uint_as_float(c == 0 ? 0x00400000u : c == 0xFFu ? 0x7FC00000u : (c << 23));
}

// rows x K of x_dtype (and r_dtype), K a multiple of 32 up to 32768; r may be null.
cudaError_t launch_rmsnorm_quantize(const void* x, int x_dtype, int64_t x_ld, const void* r,
                                    int r_dtype, int64_t r_ld, const float* w, float eps,
                                    void* r_out, int64_t o_ld, int fmt, int64_t rows, int64_t K,
                                    void* data, uint8_t* sf, cudaStream_t st);
cudaError_t launch_dequantize(int fmt, const void* data, const uint8_t* sf, int64_t outer, int64_t K,
                              void* out, int dtype, int64_t ld, cudaStream_t st);

// One tensor that mx_rope turns: tokens x heads x d, strides in elements.
struct RopeOperand {
  const uint16_t* x;
  uint16_t* y;
  long long x_ts, x_hs, y_ts, y_hs;
  int heads;
};
struct RopeCall {
  RopeOperand a, b;           // b.heads 0: there is none
  const uint64_t* freq;       // rot / 2, in 2^-64 turns a position
  const int* positions;       // one per token, or null: lens and cu
  const int* lens;
  const int* cu;
  long long tokens;
  int requests;
  int d, rot;
  int bf16;
  int neighbours;             // pairs are neighbours, else the halves' elements
  int backward;
  float factor;
};
cudaError_t launch_rope(const RopeCall& c, cudaStream_t st);

}  // namespace mxk
