// Rotary positions: pairs of channels turned by an angle that goes with the token's position,
//
//   (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t),  t = position freq  (the gradients: -t).
//
// The angle is formed in turns, as 64-bit fractions: position (freq / 2 pi 2^64) mod 2^64 by integer products.  The fraction of
// one position is off by its own last bit and, for large frequencies, by the last place of 1 / 2 pi (0.015 of it): 5 units
// of 2^-64 for |freq| < 2^10, 2^-30.7 turns at a position of 2^31.  Its upper 32 bits then go through sincospi: 2^-30 turns in all.
// 6 operations per pair on 8 bytes of 16-bit data: the bound is memory.  The sines and cosines are
// shared by a token's heads: a thread keeps those of its pairs and walks over heads.
#include "s4_block.cuh"
#include "s4_sequence.h"

namespace {
using namespace s4blk;

// freq / (2 pi) in units of 2^-64 turns, modulo 2^64, from the number's own bits: |freq| = m 2^(e - 52) with m
// below 2^53, times 2^66 / (2 pi) rounded to 64 bits.
__device__ __forceinline__ unsigned long long turns_of(double freq) {
  const unsigned long long bits = (unsigned long long)__double_as_longlong(freq);
  const int e = (int)(bits >> 52 & 0x7ff);
  const unsigned long long m = (bits & 0xfffffffffffffull) | (e ? 1ull << 52 : 0ull);
  constexpr unsigned long long kTurn = 0xa2f9836e4e44152aull;  // 2^66 / (2 pi) = 11743562013128004905.98
  const unsigned long long hi = __umul64hi(m, kTurn), lo = m * kTurn;
  const int s = 54 - ((e ? e : 1) - 1023);  // the product's bits below 2^-64 turns
  unsigned long long t;
  if (s >= 128 || s <= -64)
    t = 0;
  else if (s >= 64)
    t = hi >> (s - 64);
  else if (s > 0)
    t = hi << (64 - s) | lo >> s;
  else
    t = lo << -s;
  return bits >> 63 ? 0ull - t : t;
}

// P pairs as they lie: two packs of P (halves) or one of 2 P elements (interleaved).  P = 1 takes any
// alignment: single elements.
template <typename T, int P, bool PAIRS>
struct Turned {
  static constexpr bool ONE = PAIRS && P > 1;  // one pack of both
  Pack<T, ONE ? 2 * P : P> u, v;
  __device__ __forceinline__ void load(const T* x, int R, int i) {
    if constexpr (ONE) {
      u = ld_whole<T, 2 * P>(x + 2 * i);
    } else {
      u = ld_whole<T, P>(x + (PAIRS ? 2 * i : i));
      v = ld_whole<T, P>(x + (PAIRS ? 2 * i + 1 : R + i));
    }
  }
  __device__ __forceinline__ float a(int j) const { return ONE ? u.get(2 * j) : u.get(j); }
  __device__ __forceinline__ float b(int j) const { return ONE ? u.get(2 * j + 1) : v.get(j); }
  __device__ __forceinline__ static void store(T* x, int R, int i, const float (&a)[P], const float (&b)[P]) {
    if constexpr (ONE) {
      float w[2 * P];
#pragma unroll
      for (int j = 0; j < P; ++j) w[2 * j] = a[j], w[2 * j + 1] = b[j];
      st_whole<T, 2 * P>(x + 2 * i, w);
    } else {
      st_whole<T, P>(x + (PAIRS ? 2 * i : i), a);
      st_whole<T, P>(x + (PAIRS ? 2 * i + 1 : R + i), b);
    }
  }
};

// Heads whose channels a thread has on their way, and CTAs per SM: 4 x 4096 tokens of 32 heads of 128 channels in bfloat16 take
// 50 us (a plain copy 44); with one head or four at once 55 and 64, without the bound on registers 70
// (which spills 64 to 104 bytes a thread where halves of 16 bits go in packs of 8).
constexpr int kAtOnce = 2, kPerSm = 4;

// Threads: `units` per token and head lane (packs of P pairs, and packs of W copied channels), `lanes`
// head lanes per token, `per` tokens.  Tokens in steps of the grid.
template <typename T, int P, int W, bool PAIRS, bool COPIES>
__global__ void __launch_bounds__(256, kPerSm) rotary_kernel(s4_rotary_args a, int units, int lanes, int per) {
  // first the threads that turn, then those that copy: a warp has one kind or the other
  const int turned = COPIES ? a.R / P : units, heads = a.H + a.G, split = turned * lanes * per;
  const bool copy = COPIES && (int)threadIdx.x >= split;
  const int id = threadIdx.x - (copy ? split : 0), mine = copy ? units - turned : turned;
  if (mine == 0) return;
  const int u = id % mine, lane = id / mine % lanes, sub = id / mine / lanes;
  if (sub >= per) return;
  const int at = copy ? 2 * a.R + u * W : u * P;
  unsigned long long turn[P];
  if (!copy) {
#pragma unroll
    for (int j = 0; j < P; ++j) turn[j] = turns_of(rd(a.freqs + at + j));
  }
  const long long tokens = (long long)a.batch * a.L;
  for (long long token = (long long)blockIdx.x * per + sub; token < tokens; token += (long long)gridDim.x * per) {
    const long long b = token / a.L, t = token - b * a.L;
    const auto place = [&](int h, const T*& x, T*& y) {
      const bool query = h < a.H;
      const s4_heads& in = query ? a.q : a.k;
      const s4_heads_out& out = query ? a.q_out : a.k_out;
      const int head = query ? h : h - a.H;
      x = static_cast<const T*>(in.p) + b * in.batch + t * in.row + head * in.head;
      y = static_cast<T*>(out.p) + b * out.batch + t * out.row + head * out.head;
    };
    const T* x[kAtOnce];
    T* y[kAtOnce];
    if (copy) {
      for (int h0 = lane; h0 < heads; h0 += kAtOnce * lanes) {
        Pack<T, W> v[kAtOnce];
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (h0 + i * lanes < heads) {
            place(h0 + i * lanes, x[i], y[i]);
            if (x[i] != y[i]) v[i] = ld_whole<T, W>(x[i] + at);
          }
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i)
          if (h0 + i * lanes < heads && x[i] != y[i]) st_pack<T, W>(y[i] + at, W, true, v[i]);
      }
      continue;
    }
    // the first heads' channels are on their way before the sines and cosines are formed
    Turned<T, P, PAIRS> v[kAtOnce];
    const auto load = [&](int h0) {
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (h0 + i * lanes < heads) {
          place(h0 + i * lanes, x[i], y[i]);
          v[i].load(x[i], a.R, at);
        }
    };
    const long long pos = a.positions ? (long long)rd(a.positions + b * a.positions_batch + t) : t;
    load(lane);
    float c[P], s[P];
#pragma unroll
    for (int j = 0; j < P; ++j) {
      // the signed fraction of a turn, in half turns
      const unsigned long long f = (unsigned long long)pos * turn[j];
      sincospif((float)(int)(f >> 32) * 0x1p-31f, &s[j], &c[j]);
      s[j] *= a.inverse ? -a.amplitude : a.amplitude;
      c[j] *= a.amplitude;
    }
    for (int h0 = lane; h0 < heads; h0 += kAtOnce * lanes) {
      if (h0 != lane) load(h0);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (h0 + i * lanes >= heads) continue;
        float p[P], q[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float e = v[i].a(j), f = v[i].b(j);
          p[j] = e * c[j] - f * s[j];
          q[j] = e * s[j] + f * c[j];
        }
        Turned<T, P, PAIRS>::store(y[i], a.R, at, p, q);
      }
    }
  }
}

template <typename T, int P, int W, bool PAIRS>
cudaError_t launch(const s4_rotary_args& a, cudaStream_t s) {
  const int units = a.R / P + (a.D - 2 * a.R) / W, heads = a.H + a.G;
  const long long tokens = (long long)a.batch * a.L;
  // A thread takes up to 8 heads of its token, and fewer where that leaves the GPU idle.
  int lanes = heads;
  for (int each : {8, 4, 2}) {
    const int n = (heads + each - 1) / each;
    if (tokens * n * units >= (long long)s4impl::num_sms() * 1024) {
      lanes = n;
      break;
    }
  }
  if (lanes * units > 256) lanes = 256 / units > 0 ? 256 / units : 1;
  const int per = 256 / (lanes * units) > 0 ? 256 / (lanes * units) : 1;
  const long long need = (tokens + per - 1) / per, most = (long long)s4impl::num_sms() * 16;
  s4impl::TimedLaunch tl("rotary", s);
  const unsigned grid = (unsigned)(need < most ? need : most), threads = (units * lanes * per + 31) / 32 * 32;
  if (a.D == 2 * a.R)
    rotary_kernel<T, P, W, PAIRS, false><<<grid, threads, 0, s>>>(a, units, lanes, per);
  else
    rotary_kernel<T, P, W, PAIRS, true><<<grid, threads, 0, s>>>(a, units, lanes, per);
  return cudaGetLastError();
}

// Whether packs of `n` elements of `e` bytes fit the strides and addresses of all arrays.
bool packs_ok(const s4_rotary_args& a, int e, int n) {
  const auto ok = [&](const auto& r) { return vec_ok(r.p, e, e * n, r.batch, r.row) && vec_ok(r.p, e, e * n, r.head); };
  return ok(a.q) && ok(a.k) && ok(a.q_out) && ok(a.k_out);
}

template <typename T, bool PAIRS>
cudaError_t with_packs(const s4_rotary_args& a, cudaStream_t s) {
  constexpr int e = sizeof(T), most = 16 / e;
  const int tail = a.D - 2 * a.R;
  // one pack is 16 bytes where the heads allow it (P pairs: P channels of each half, or 2 P interleaved)
  constexpr int P = PAIRS ? most / 2 : most;
  const int units = a.R / P + tail / most;
  if (a.R % P == 0 && (PAIRS ? 2 * a.R % most == 0 : true) && tail % most == 0 && units >= 1 && units <= 256 &&
      packs_ok(a, e, most))
    return launch<T, P, most, PAIRS>(a, s);
  // pair by pair, element by element (4 x 4096 tokens of 32 heads of 128 channels in bfloat16: 49 us in packs, 134 at an odd
  // address, 176 with 126 channels turned)
  return launch<T, 1, 1, PAIRS>(a, s);
}

template <typename T>
cudaError_t with_layout(const s4_rotary_args& a, cudaStream_t s) {
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  const int e = sizeof(T);
  const auto add = [&](const auto& r, int heads, bool write) {
    x.add(r.p, e, !write, write, a.D, a.batch, r.batch, a.L, r.row, heads, r.head);
  };
  add(a.q, a.H, false), add(a.k, a.G, false), add(a.q_out, a.H, true), add(a.k_out, a.G, true);
  x.in(a.freqs, 8, a.R);
  x.add(a.positions, 4, true, false, a.L, a.batch, a.positions_batch);
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  return a.pairs ? with_packs<T, true>(a, s) : with_packs<T, false>(a, s);
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_rotary)
#endif

cudaError_t launch_rotary(const s4_rotary_args& a, cudaStream_t s) {
  if (a.dtype == S4_F32) return with_layout<float>(a, s);
  return a.dtype == S4_BF16 ? with_layout<__nv_bfloat16>(a, s) : with_layout<__half>(a, s);
}

}  // namespace s4impl
