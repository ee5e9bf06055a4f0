// Shared by the selective scan's kernels (forward, single token, backward): how a CTA's threads
// map to channels and states, the tiles it stages and the sums over lanes.
//
// A channel's N states lie on LPC neighbouring lanes of a warp, SPT consecutive states each
// (N <= LPC SPT, the rest padded with zeros); a thread serves CPT consecutive channels.  All
// channels of a CTA belong to one group of B and C.
#pragma once
#include "s4_block.cuh"

namespace s4sel {
using namespace s4blk;
using s4impl::St;

constexpr int kThreads = 128;
constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

// 2^v (relative error 2^-22, 0 for results below the normal range)
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// log(1 + e^v) without overflow and with its relative precision for very negative v
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v))); }

// A CTA's channels: blocks of HB within a group.
struct Chan {
  int g, h0, hend;  // group, first channel, end of the group's channels
};
template <int HB>
__device__ __forceinline__ Chan chan_of(int block, int Hg) {
  const int per = (Hg + HB - 1) / HB;
  Chan c;
  c.g = block / per;
  c.h0 = c.g * Hg + (block % per) * HB;
  c.hend = (c.g + 1) * Hg;
  return c;
}

// [TT][NP] of B or C in fp32, tokens from t0 (those from `len` on, and padded states, as zeros).
template <typename T, int TT, int NP>
__device__ __forceinline__ void stage_vectors(float* s, const T* p, long long row, int t0, int len, int N) {
  for (int i = threadIdx.x; i < TT * NP; i += kThreads) {
    const int t = i / NP, n = i % NP;
    s[i] = t0 + t < len && n < N ? to_f(p[(t0 + t) * row + n]) : 0.f;
  }
}

// Four tokens' values v[0..3] of a channel, summed over its LPC lanes.  With LPC >= 4 the lane
// comes to hold the sum of token (lane & 3), after 3 exchanges rather than 8; with fewer lanes
// each holds 4 / LPC tokens (v[0] .. for tokens own, own + LPC ...).
template <int LPC>
__device__ __forceinline__ void sum_lanes(float (&v)[4], int lane) {
  if constexpr (LPC >= 2) {
    const bool b = lane & 1;
    float k0 = b ? v[1] : v[0], s0 = b ? v[0] : v[1];
    float k1 = b ? v[3] : v[2], s1 = b ? v[2] : v[3];
    v[0] = k0 + __shfl_xor_sync(0xffffffffu, s0, 1);
    v[1] = k1 + __shfl_xor_sync(0xffffffffu, s1, 1);
  }
  if constexpr (LPC >= 4) {
    const bool b = lane & 2;
    const float k = b ? v[1] : v[0], s = b ? v[0] : v[1];
    v[0] = k + __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
    for (int o = 4; o < LPC; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  }
}
// Tokens (of four) a lane holds after sum_lanes, and the i-th of them.
template <int LPC>
constexpr int kOwn = LPC >= 4 ? 1 : 4 / LPC;
template <int LPC>
__device__ __forceinline__ int own_token(int lane, int i) {
  return LPC >= 4 ? (lane & 3) : (lane & (LPC - 1)) + i * LPC;
}

}  // namespace s4sel
