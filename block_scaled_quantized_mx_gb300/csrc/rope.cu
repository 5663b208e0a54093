// rope.cu -- rotary positions of queries and keys.
//
//   (u, w) = f * (a cos t - b sin t, a sin t + b cos t),  t = position * freq_i
// for the pairs (a, b) of a head's first `rot` values: elements i and i + rot / 2, or
// neighbours 2 i and 2 i + 1; the rest of the head goes through as it is.  backward:
// the transposed map, t negated, for gradients.
//
// Angles.  A frequency is a number of turns for each position, kept as a whole
// number of 2^-64 turns: position * freq in 64 bits that wrap is then the angle
// modulo one turn, exactly, at any position (of freq itself 2^-65 turns are lost, at
// position 2^31 2^-34).  What is left is in [-1/2, 1/2) turns, where fp32 serves.
//
// Bound: HBM, each value read and written once.  Cosines and sines are computed
// once per token for all heads and both operands, into shared memory; the values' loads
// are on their way meanwhile.  A token's request is found in cu by a warp, 32
// offsets a step.
#include <cstdint>

#include "common.cuh"
#include "layer_common.cuh"
#include "ptx.cuh"

namespace mxk {

namespace {

constexpr int RP_THREADS = 256;
constexpr int RP_MOST_TOKENS = 4;           // of a CTA
constexpr int RP_BATCH = 4;                 // units whose loads are in flight together
constexpr int RP_MOST_ROT = 512;

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

// A unit is two chunks of 8 values of one head: turned, (8 u, 8 u + rot / 2) or
// 16 consecutive; or behind them 16 (or the last 8) that go through.
struct RopeUnit {
  const uint16_t* x;
  uint16_t* y;
  int first, second;          // elements; second < 0: there is none
  int u;                      // among the head's turned units; -1: goes through
};

template <int TOKENS>
__global__ void __launch_bounds__(RP_THREADS) rope_kernel(const RopeCall c) {
  __shared__ float2 sm_turn[TOKENS * (RP_MOST_ROT / 2)];
  __shared__ int sm_pos[TOKENS];
  __shared__ int sm_live[TOKENS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long t0 = static_cast<long long>(blockIdx.x) * TOKENS;
  const int turned = c.rot / 16, per_head = turned + (c.d - c.rot + 15) / 16;
  const int per_token = (c.a.heads + c.b.heads) * per_head;
  const int tokens = static_cast<int>(min(static_cast<long long>(TOKENS), c.tokens - t0));
  const int units = tokens * per_token;
  auto unit = [&](int i) {
    RopeUnit r;
    const int token = i / per_token, rest = i - token * per_token;
    const int head = rest / per_head, u = rest - head * per_head;
    const bool of_b = head >= c.a.heads;
    const RopeOperand& o = of_b ? c.b : c.a;
    const int h = of_b ? head - c.a.heads : head;
    r.x = o.x + (t0 + token) * o.x_ts + h * o.x_hs;
    r.y = o.y + (t0 + token) * o.y_ts + h * o.y_hs;
    if (u < turned) {
      r.u = u;
      r.first = c.neighbours ? 16 * u : 8 * u;
      r.second = c.neighbours ? 16 * u + 8 : 8 * u + c.rot / 2;
    } else {
      r.u = -1;
      r.first = c.rot + 16 * (u - turned);
      r.second = r.first + 8 < c.d ? r.first + 8 : -1;
    }
    return r;
  };
  uint4 va[RP_BATCH], vb[RP_BATCH];
  auto load = [&](int i0) {
#pragma unroll
    for (int k = 0; k < RP_BATCH; ++k) {
      const int i = i0 + k * RP_THREADS;
      if (i >= units) break;
      const RopeUnit r = unit(i);
      va[k] = *reinterpret_cast<const uint4*>(r.x + r.first);
      if (r.second >= 0) vb[k] = *reinterpret_cast<const uint4*>(r.x + r.second);
    }
  };
  load(tid);
  for (int t = warp; t < tokens; t += RP_THREADS / 32) {
    int pos = 0;
    const bool live = rope_position(c, t0 + t, lane, pos);
    if (lane == 0) {
      sm_pos[t] = pos;
      sm_live[t] = live;
    }
  }
  __syncthreads();
  const int pairs = c.rot / 2;
  for (int i = tid; i < tokens * pairs; i += RP_THREADS) {
    const int t = i / pairs;
    const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(sm_pos[t])) * c.freq[i - t * pairs];
    float s, co;
    sincospif(static_cast<float>(static_cast<int64_t>(turn)) * 1.0842021724855044e-19f, &s, &co);   // 2^-63
    sm_turn[i] = make_float2(co * c.factor, (c.backward ? -s : s) * c.factor);
  }
  __syncthreads();
  for (int i0 = tid; i0 < units; i0 += RP_BATCH * RP_THREADS) {
    if (i0 != tid) load(i0);
#pragma unroll
    for (int k = 0; k < RP_BATCH; ++k) {
      const int i = i0 + k * RP_THREADS;
      if (i >= units) break;
      const int token = i / per_token;
      if (!sm_live[token]) continue;         // belongs to no request: left as it is
      const RopeUnit r = unit(i);
      if (r.u < 0) {
        if (r.x != r.y) {
          *reinterpret_cast<uint4*>(r.y + r.first) = va[k];
          if (r.second >= 0) *reinterpret_cast<uint4*>(r.y + r.second) = vb[k];
        }
        continue;
      }
      const float2* turn = sm_turn + token * pairs + 8 * r.u;
      uint32_t p[4] = {va[k].x, va[k].y, va[k].z, va[k].w}, q[4] = {vb[k].x, vb[k].y, vb[k].z, vb[k].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float a0, a1, b0, b1;
        unpack16x2(p[e], c.bf16, a0, a1);
        unpack16x2(q[e], c.bf16, b0, b1);
        if (c.neighbours) {
          const float2 s = turn[e], z = turn[4 + e];
          p[e] = pack16x2(a0 * s.x - a1 * s.y, a0 * s.y + a1 * s.x, c.bf16);
          q[e] = pack16x2(b0 * z.x - b1 * z.y, b0 * z.y + b1 * z.x, c.bf16);
        } else {
          const float2 s = turn[2 * e], z = turn[2 * e + 1];
          p[e] = pack16x2(a0 * s.x - b0 * s.y, a1 * z.x - b1 * z.y, c.bf16);
          q[e] = pack16x2(a0 * s.y + b0 * s.x, a1 * z.y + b1 * z.x, c.bf16);
        }
      }
      *reinterpret_cast<uint4*>(r.y + r.first) = make_uint4(p[0], p[1], p[2], p[3]);
      *reinterpret_cast<uint4*>(r.y + r.second) = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeCall& c, cudaStream_t st) {
  // a token to a CTA where that leaves no SM with more than a few
  if (c.tokens <= 4 * 152) {
    rope_kernel<1><<<static_cast<unsigned>(c.tokens), RP_THREADS, 0, st>>>(c);
  } else {
    const long long ctas = (c.tokens + RP_MOST_TOKENS - 1) / RP_MOST_TOKENS;
    rope_kernel<RP_MOST_TOKENS><<<static_cast<unsigned>(ctas), RP_THREADS, 0, st>>>(c);
  }
  return cudaGetLastError();
}

}  // namespace mxk
