// Rotary positions: pairs of channels turned by an angle that goes with the token's position,
//
//   (a, b) -> amplitude (a cos t - b sin t, a sin t + b cos t),  t = position freq  (the gradients: -t).
//
// The angle is formed in turns, as 64-bit fractions: position (freq / 2 pi 2^64) mod 2^64 by integer products is
// exact but for the fraction's own last bit, at any position; its upper 32 bits then go through sincospi.
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
__device__ __forceinline__ void ld_pairs_of(const T* x, int R, int i, float (&a)[P], float (&b)[P]) {
  if constexpr (PAIRS && P == 1) {
    a[0] = to_f(rd(x + 2 * i)), b[0] = to_f(rd(x + 2 * i + 1));
  } else if constexpr (PAIRS) {
    const Pack<T, 2 * P> v = ld_whole<T, 2 * P>(x + 2 * i);
#pragma unroll
    for (int j = 0; j < P; ++j) a[j] = v.get(2 * j), b[j] = v.get(2 * j + 1);
  } else {
    const Pack<T, P> u = ld_whole<T, P>(x + i), v = ld_whole<T, P>(x + R + i);
#pragma unroll
    for (int j = 0; j < P; ++j) a[j] = u.get(j), b[j] = v.get(j);
  }
}
template <typename T, int P, bool PAIRS>
__device__ __forceinline__ void st_pairs_of(T* x, int R, int i, const float (&a)[P], const float (&b)[P]) {
  if constexpr (PAIRS && P == 1) {
    wr(x + 2 * i, from_f<T>(a[0])), wr(x + 2 * i + 1, from_f<T>(b[0]));
  } else if constexpr (PAIRS) {
    float v[2 * P];
#pragma unroll
    for (int j = 0; j < P; ++j) v[2 * j] = a[j], v[2 * j + 1] = b[j];
    st_whole<T, 2 * P>(x + 2 * i, v);
  } else {
    st_whole<T, P>(x + i, a);
    st_whole<T, P>(x + R + i, b);
  }
}

// Threads: `units` per token and head lane (packs of P pairs, then packs of W copied channels), `lanes`
// head lanes per token, tokens.  Tokens in steps of the grid.
template <typename T, int P, int W, bool PAIRS>
__global__ void __launch_bounds__(256) rotary_kernel(s4_rotary_args a, int units, int lanes, int per) {
  const int u = threadIdx.x % units, rest = threadIdx.x / units, lane = rest % lanes, sub = rest / lanes;
  if (sub >= per) return;
  const int turned = (a.R + P - 1) / P, heads = a.H + a.G;
  const bool copy = u >= turned;
  const int at = copy ? 2 * a.R + (u - turned) * W : u * P;
  unsigned long long turn[P];
  if (!copy) {
#pragma unroll
    for (int j = 0; j < P; ++j) turn[j] = turns_of(rd(a.freqs + at + j));
  }
  const long long tokens = (long long)a.batch * a.L;
  for (long long token = (long long)blockIdx.x * per + sub; token < tokens; token += (long long)gridDim.x * per) {
    const long long b = token / a.L, t = token - b * a.L;
    float c[P], s[P];
    if (!copy) {
      const long long pos = a.positions ? (long long)rd(a.positions + b * a.positions_batch + t) : t;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        // the signed fraction of a turn, in half turns
        const unsigned long long f = (unsigned long long)pos * turn[j];
        sincospif((float)(int)(f >> 32) * 0x1p-31f, &s[j], &c[j]);
        s[j] *= a.inverse ? -a.amplitude : a.amplitude;
        c[j] *= a.amplitude;
      }
    }
#pragma unroll 4
    for (int h = lane; h < heads; h += lanes) {
      const bool query = h < a.H;
      const s4_heads& in = query ? a.q : a.k;
      const s4_heads_out& out = query ? a.q_out : a.k_out;
      const int head = query ? h : h - a.H;
      const T* x = static_cast<const T*>(in.p) + b * in.batch + t * in.row + head * in.head;
      T* y = static_cast<T*>(out.p) + b * out.batch + t * out.row + head * out.head;
      if (copy) {
        if (x != y) st_pack<T, W>(y + at, W, true, ld_whole<T, W>(x + at));
        continue;
      }
      float p[P], q[P];
      ld_pairs_of<T, P, PAIRS>(x, a.R, at, p, q);
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float v = p[j] * c[j] - q[j] * s[j];
        q[j] = p[j] * s[j] + q[j] * c[j];
        p[j] = v;
      }
      st_pairs_of<T, P, PAIRS>(y, a.R, at, p, q);
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
  rotary_kernel<T, P, W, PAIRS><<<(unsigned)(need < most ? need : most), (units * lanes * per + 31) / 32 * 32, 0, s>>>(
      a, units, lanes, per);
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
