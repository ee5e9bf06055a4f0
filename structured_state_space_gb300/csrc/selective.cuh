// Shared by the selective scan's kernels (forward, single token, backward): how a CTA's threads
// map to channels and states, activations, packed arithmetic and the sums over lanes.
//
// A channel's N states lie on LPC neighbouring lanes of a warp, SPT consecutive states each
// (N <= LPC SPT, the rest padded with zeros).  A thread serves several neighbouring channels.  Packed
// fp32 operations issue two multiplications or additions at once (the rate of 128 a clock per
// SM is the same: packing saves issue slots, not arithmetic).  All channels of a warp or CTA
// that works together belong to one group of B and C.
#pragma once
#include "s4_block.cuh"

namespace s4sel {
using namespace s4blk;
using s4impl::St;

constexpr int kThreads = 128;
constexpr float kLn2 = 0.69314718055994530942f;

// ---- functions ----------------------------------------------------------------------------
// log(1 + e^v) = max(v, 0) + log1p(u), u = e^-|v|: no overflow, and the relative precision of
// log1p for small u.  log1p(u) = 2 atanh(s) with s = u / (2 + u) <= 1/3; 2 atanh(s) / s is a
// polynomial in s^2 on [0, 1/9], here its interpolation at the Chebyshev points of degree 4
// (relative error 8e-9, below the rounding of s).
__device__ __forceinline__ float softplus(float v) {
  const float u = ex2(-fabsf(v) * kLog2e), s = u * s4dev::rcp_approx(2.f + u), q = s * s;
  float p = 0.2817465662956238f;
  p = fmaf(p, q, 0.2796141803264618f);
  p = fmaf(p, q, 0.40024852752685547f);
  p = fmaf(p, q, 0.6666631698608398f);
  p = fmaf(p, q, 2.f);
  return fmaf(s, p, fmaxf(v, 0.f));
}
// The same of a pair, in packed operations.
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 u = make_float2(ex2(-fabsf(v.x) * kLog2e), ex2(-fabsf(v.y) * kLog2e));
  const float2 two = make_float2(2.f, 2.f), w = add2(u, two);
  const float2 s = mul2(u, make_float2(s4dev::rcp_approx(w.x), s4dev::rcp_approx(w.y))), q = mul2(s, s);
  float2 p = fma2(make_float2(0.2817465662956238f, 0.2817465662956238f), q,
                  make_float2(0.2796141803264618f, 0.2796141803264618f));
  p = fma2(p, q, make_float2(0.40024852752685547f, 0.40024852752685547f));
  p = fma2(p, q, make_float2(0.6666631698608398f, 0.6666631698608398f));
  p = fma2(p, q, two);
  return fma2(s, p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// Rows of shared memory, one per token, of one VEC-float vector per channel slot: the floats to add
// to `row` of them so that the LPC tokens and the slots that a warp writes at once (8 lanes of 16
// bytes, 16 of 8) lie in different banks.
constexpr int row_pad(int lpc, int row) { return lpc == 1 ? 0 : lpc <= 4 ? (32 / lpc + 32 - row % 32) % 32 : 8; }

// A CTA's channels: blocks of HB within a group.
struct Chan {
  int g, h0, hend;  // group, first channel, end of the group's channels
};
template <int HB>
__host__ __device__ __forceinline__ int chan_blocks(int H, int G) {
  return G * ((H / G + HB - 1) / HB);
}
template <int HB>
__device__ __forceinline__ Chan chan_of(int block, int Hg) {
  const int per = (Hg + HB - 1) / HB;
  Chan c;
  c.g = block / per;
  c.h0 = c.g * Hg + (block % per) * HB;
  c.hend = (c.g + 1) * Hg;
  return c;
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
