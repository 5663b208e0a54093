// rope.cu -- rotary positions of queries and keys.
//
//   (u, w) = f * (a cos t - b sin t, a sin t + b cos t),  t = position * freq_i
// for the pairs (a, b) of a head's first `rot` values: elements i and i + rot / 2, or
// neighbours 2 i and 2 i + 1; the rest of the head goes through as it is.  backward:
// the transposed map, t negated, for gradients.
//
// Angles.  A frequency is a number of turns for each position, kept as a whole
// number of 2^-64 turns: position * freq in 64 bits that wrap is then the angle
// modulo one turn, exactly, at any position.  (Of a frequency itself 2^-65 turns are lost where
// freq is the nearest whole number; mx.rope_frequencies computes in doubles, within 2^-52 turns, at
// position 2^20 2^-32, at 2^31 2^-21.)  What is left is in [-1/2, 1/2) turns, where fp32 serves.
//
// Bound: HBM, each value read and written once.  Cosines and sines are computed
// once per token for all heads and both operands, into shared memory; the values' loads
// are on their way meanwhile.  A token's request is found in cu by a warp, 32
// offsets a step.
// Measured, 32 + 8 heads of 128: 8192 tokens 30 us, 5.6 TB/s, 0.82 of the copy rate, 17000
// tokens 57 us, 0.90: what is left is the wait for the tokens' positions, three reads from L2
// one after the other, before the first value is turned; 64 tokens 2.4 us.  (A thread with 2,
// 3, 4 and 8 tokens: 8192 tokens 31.7, 30.0, 32.1 and 44 us, 17000 60.8, 56.9 and 58.5; a grid
// that stays, with three tokens ahead, 31.9, and small calls slower; a request's offset, end and
// length read together 20.0 -> 19.7 at 4800 tokens but 56.9 -> 59.2 at 17000.)
#include <cstdint>

#include "common.cuh"
#include "layer_common.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int RP_MOST_THREADS = 512;
constexpr int RP_TOKENS = 3;                // of a thread, where there are many
constexpr int RP_SMEM = 32768;              // cosines and sines of a CTA at the most

// The position of token t, found by a whole warp; false: it belongs to no request.
__device__ __forceinline__ bool rope_position(const RopeCall& c, long long t, int lane, int& pos) {
  if (c.positions != nullptr) {
    pos = c.positions[t];
    return true;
  }
  int lo = 0, n = c.requests;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const bool begun = lane * step < n && c.cu[lo + lane * step] <= t;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, begun));
    if (k == 0) return false;
    lo += (k - 1) * step;
    n = step == 1 ? 0 : min(step, n - (k - 1) * step);
  }
  const int end = c.cu[lo + 1];
  pos = c.lens[lo] - static_cast<int>(end - t);
  return t < end;
}

__device__ __forceinline__ uint32_t pack16x2(float lo, float hi, int bf16) {
  return bf16 ? cvt_bf16x2(lo, hi) : cvt_f16x2(lo, hi);
}

// A unit is two chunks of 8 values of one head: turned, elements 8 u .. and 8 u +
// rot / 2 .., or 16 consecutive ones; or behind them 16 (or the last 8) that go
// through.  A thread takes the same unit of TOKENS tokens, their loads together: its
// place in the head and the heads' strides are worked out once.  `sets` such groups
// of tokens make a CTA where a token has few units.
// Cosines and sines stand in shared memory as the units read them: two pairs' to 16
// bytes, pairs 2 e and 2 e + 1 of unit u of a token at [e][u], so that a warp's
// reads are consecutive.
struct RopeShape {
  int units;                  // of a token
  int per_head;
  int threads;                // of a set
  int sets;
};

template <int TOKENS>
__global__ void __launch_bounds__(RP_MOST_THREADS, 2) rope_kernel(const RopeCall c, const RopeShape z) {
  extern __shared__ float4 sm_turn[];       // [tokens of the CTA][4][turned units]
  __shared__ int sm_pos[RP_MOST_THREADS];
  __shared__ int sm_live[RP_MOST_THREADS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const int turned = c.rot / 16;
  const long long t0 = static_cast<long long>(blockIdx.x) * (TOKENS * z.sets);
  const int tokens = static_cast<int>(min(static_cast<long long>(TOKENS * z.sets), c.tokens - t0));
  const int set = tid / z.threads, in_set = tid - set * z.threads;
  const int mine = set < z.sets ? min(TOKENS, tokens - TOKENS * set) : 0;   // (0 or less: none)
  const uint16_t* x;
  uint16_t* y;
  long long x_ts, y_ts;
  int first, second, u;                     // elements (second < 0: there is none); u < 0: goes through
  auto enter = [&](int i) {
    const int head = i / z.per_head;
    u = i - head * z.per_head;
    const bool of_b = head >= c.a.heads;
    const RopeOperand& o = of_b ? c.b : c.a;
    const int h = of_b ? head - c.a.heads : head;
    x_ts = o.x_ts;
    y_ts = o.y_ts;
    x = o.x + (t0 + TOKENS * set) * x_ts + h * o.x_hs;
    y = o.y + (t0 + TOKENS * set) * y_ts + h * o.y_hs;
    if (u < turned) {
      first = c.neighbours ? 16 * u : 8 * u;
      second = c.neighbours ? 16 * u + 8 : 8 * u + c.rot / 2;
    } else {
      first = c.rot + 16 * (u - turned);
      second = first + 8 < c.d ? first + 8 : -1;
      u = -1;
    }
  };
  wait_for_stream();
  uint4 va[TOKENS], vb[TOKENS];
  auto load = [&] {
#pragma unroll
    for (int t = 0; t < TOKENS; ++t)
      if (t < mine) {
        va[t] = *reinterpret_cast<const uint4*>(x + t * x_ts + first);
        if (second >= 0) vb[t] = *reinterpret_cast<const uint4*>(x + t * x_ts + second);
      }
  };
  if (in_set < z.units) {
    enter(in_set);
    load();
  }
  for (int t = warp; t < tokens; t += warps) {
    int pos = 0;
    const bool live = rope_position(c, t0 + t, lane, pos);
    if (lane == 0) {
      sm_pos[t] = pos;
      sm_live[t] = live;
    }
  }
  __syncthreads();
  const int pairs = c.rot / 2;
  for (int i = tid; i < tokens * pairs; i += blockDim.x) {
    const int t = i / pairs, p = i - t * pairs;
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(sm_pos[t])) * c.freq[p];
    float s, co;
    sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 1.0842021724855044e-19f, &s, &co);   // 2^-63
    reinterpret_cast<float2*>(sm_turn)[2 * ((4 * t + ((p & 7) >> 1)) * turned + (p >> 3)) + (p & 1)] =
        make_float2(co * c.factor, (c.backward ? -s : s) * c.factor);
  }
  __syncthreads();
  for (int i = in_set; i < z.units; i += z.threads) {
    if (i != in_set) {
      enter(i);
      load();
    }
#pragma unroll
    for (int t = 0; t < TOKENS; ++t) {
      if (t >= mine || !sm_live[TOKENS * set + t]) continue;   // of no request: left as it is
      uint16_t* to = y + t * y_ts;
      if (u < 0) {
        if (x != y) {
          *reinterpret_cast<uint4*>(to + first) = va[t];
          if (second >= 0) *reinterpret_cast<uint4*>(to + second) = vb[t];
        }
        continue;
      }
      const float4* turn = sm_turn + 4 * (TOKENS * set + t) * turned + u;
      uint32_t p[4] = {va[t].x, va[t].y, va[t].z, va[t].w}, q[4] = {vb[t].x, vb[t].y, vb[t].z, vb[t].w};
      float a[8], b[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        unpack16x2(p[e], c.bf16, a[2 * e], a[2 * e + 1]);
        unpack16x2(q[e], c.bf16, b[2 * e], b[2 * e + 1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 s = turn[e * turned];  // of pairs 2 e and 2 e + 1
        if (c.neighbours) {
          float* v = e < 2 ? a + 4 * e : b + 4 * (e - 2);
          const float u0 = v[0] * s.x - v[1] * s.y, w0 = v[0] * s.y + v[1] * s.x;
          const float u1 = v[2] * s.z - v[3] * s.w, w1 = v[2] * s.w + v[3] * s.z;
          v[0] = u0;
          v[1] = w0;
          v[2] = u1;
          v[3] = w1;
        } else {
          const float u0 = a[2 * e] * s.x - b[2 * e] * s.y, u1 = a[2 * e + 1] * s.z - b[2 * e + 1] * s.w;
          b[2 * e] = a[2 * e] * s.y + b[2 * e] * s.x;
          b[2 * e + 1] = a[2 * e + 1] * s.w + b[2 * e + 1] * s.z;
          a[2 * e] = u0;
          a[2 * e + 1] = u1;
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = pack16x2(a[2 * e], a[2 * e + 1], c.bf16);
        q[e] = pack16x2(b[2 * e], b[2 * e + 1], c.bf16);
      }
      *reinterpret_cast<uint4*>(to + first) = make_uint4(p[0], p[1], p[2], p[3]);
      *reinterpret_cast<uint4*>(to + second) = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, cudaStream_t st) {
  RopeShape z;
  const int turned = c.rot / 16;
  z.per_head = turned + (c.d - c.rot + 15) / 16;
  const long long units = static_cast<long long>(c.a.heads + c.b.heads) * z.per_head;
  z.units = static_cast<int>(units);
  // a token's units in as few equal rounds as there must be
  const long long rounds = (units + RP_MOST_THREADS - 1) / RP_MOST_THREADS;
  z.threads = static_cast<int>((units + rounds - 1) / rounds);
  // one token a thread where three would leave SMs idle
  const bool many = c.tokens > 4 * 152;
  const int per = many ? RP_TOKENS : 1;
  const int fits = RP_SMEM / (per * turned * 64);
  z.sets = 1;
  if (many) {
    z.sets = 256 / z.threads;
    if (z.sets > fits) z.sets = fits;
    if (z.sets < 1) z.sets = 1;
  }
  const int threads = (z.threads * z.sets + 31) / 32 * 32;
  const long long of_cta = static_cast<long long>(per) * z.sets;
  const unsigned ctas = static_cast<unsigned>((c.tokens + of_cta - 1) / of_cta);
  const size_t smem = static_cast<size_t>(of_cta) * turned * 64;
  if (many)
    return launch_early(rope_kernel<RP_TOKENS>, ctas, threads, smem, 1, st, c, z);
  return launch_early(rope_kernel<1>, ctas, threads, smem, 1, st, c, z);
}

}  // namespace mxk
