// The short causal convolution along time with SiLU, forward (prompts and single
// tokens) and backward.
//
//   v_t = bias + sum_{k<W} w[k] x[t-W+1+k],  y = v sigmoid(v)
//
// About 2 W + 5 operations on 4 bytes (16-bit types) moved: the bound is memory.  A thread
// owns V neighbouring channels and walks a segment of the sequence with the last taps in
// registers, so that each input is read from memory once and W - 1 more times per segment
// from cache.  Channels go through packed fp32 operations in pairs.
//
// Measured (bfloat16, 4 taps, 8 sequences of 4096 tokens, 2048 channels): forward 60 us (4.5 TB/s), backward 102
// us (3.9 TB/s; 29 instructions per element, half of the issue slots).
#include "s4_block.cuh"

namespace {
using namespace s4blk;
using s4impl::St;

constexpr int kSegFwd = 16;   // tokens of a thread's segment, forward
constexpr int kSegBwd = 64;   // and backward (128: the same)
constexpr int kThreads = 128;
constexpr int kWarpsBwd = 8, kVecBwd = 4;

template <typename T, int KW, int V>
__global__ void __launch_bounds__(kThreads) short_conv_kernel(s4_short_conv_args a, bool vec, St st) {
  record_gen(st);
  const int b = blockIdx.y;
  const int ncv = (a.H + V - 1) / V, nseg = (a.L + kSegFwd - 1) / kSegFwd;
  const Seq q = seq_of(a.lengths, a.index, b, a.L, a.slots, st);
  const long long gid = (long long)blockIdx.x * kThreads + threadIdx.x;
  if (gid >= (long long)ncv * nseg) return;
  const int seg = (int)(gid / ncv), h = (int)(gid % ncv) * V, n = min(V, a.H - h);
  const int t0 = seg * kSegFwd, t1 = min(a.L, t0 + kSegFwd), live = min(t1, q.len);
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
  T* y = static_cast<T*>(a.y.p) + b * a.y.batch + h;
  const long long srow = a.H, sslot = (long long)(a.W - 1) * a.H;
  const T* state = a.state ? static_cast<const T*>(a.state) + (q.slot < 0 ? 0 : q.slot) * sslot + h : nullptr;
  const bool whole = vec && n >= V;

  // the segment's first inputs, on their way before the filter is read
  Pack<T, V> in[KW];
  const auto fetch = [&](int t) {
    if (whole && t + KW <= live) {
#pragma unroll
      for (int u = 0; u < KW; ++u) in[u] = ld_whole<T, V>(x + (t + u) * a.x.row);
      return;
    }
#pragma unroll
    for (int u = 0; u < KW; ++u)
      in[u] = ld_pack<T, V>(x + (t + u) * a.x.row, t + u < live ? n : 0, vec);
  };
  if (t0 < live) fetch(t0);
  float2 w[KW][V / 2], bias[V / 2], win[KW][V / 2];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool on = i < n;
    (i % 2 ? bias[i / 2].y : bias[i / 2].x) = a.bias && on ? rd(a.bias + h + i) : 0.f;
#pragma unroll
    for (int k = 0; k < KW; ++k)
      (i % 2 ? w[k][i / 2].y : w[k][i / 2].x) = on ? rd(a.w + (long long)(h + i) * KW + k) : 0.f;
  }
  // the inputs before the segment: of the sequence, of the state, or zeros
#pragma unroll
  for (int k = 0; k < KW - 1; ++k) {
    const int t = t0 - (KW - 1) + k;
    Pack<T, V> r;
    r.zero();
    if (t >= 0 && t < q.len)
      r = ld_pack<T, V>(x + t * a.x.row, n, vec);
    else if (t < 0 && t >= -(a.W - 1) && state && q.slot >= 0)
      r = ld_pack<T, V>(state + (t + a.W - 1) * srow, n, vec);
    to_pairs<T, V>(r, win[k]);
  }
  for (int t = t0; t < live; t += KW) {
    Pack<T, V> now[KW];
#pragma unroll
    for (int u = 0; u < KW; ++u) now[u] = in[u];
    if (t + KW < live) fetch(t + KW);
#pragma unroll
    for (int u = 0; u < KW; ++u) {
      if (t + u >= live) break;
      // the window is a ring: the input of token t + u replaces that of t + u - KW
      to_pairs<T, V>(now[u], win[(KW - 1 + u) % KW]);
      float2 out[V / 2];
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        float2 v = bias[i];
#pragma unroll
        for (int k = 0; k < KW; ++k) v = fma2(w[k][i], win[(k + u) % KW][i], v);
        out[i] = a.silu ? silu(v) : v;
      }
      st_pairs<T, V>(y + (t + u) * a.y.row, n, vec, out);
    }
  }
  for (int t = max(t0, live); t < t1; ++t) {  // padding
    const float zero[V] = {};
    st_f<T, V>(y + t * a.y.row, n, vec, zero);
  }
  // The state after the last real token, row j being input len - (W-1) + j.  The thread
  // that read the channels' old state writes the new one (in place too: rows are taken
  // from rows at or after them, in ascending order).  A single token is taken from its
  // register: y may be x there, and has been written.
  if (seg == 0 && a.state_out && q.slot >= 0) {
    T* so = static_cast<T*>(a.state_out) + q.slot * sslot + h;
    for (int j = 0; j < a.W - 1; ++j) {
      const int t = q.len - (a.W - 1) + j;
      Pack<T, V> r;
      r.zero();
      if (t >= 0)
        r = a.L == 1 ? in[0] : ld_pack<T, V>(x + t * a.x.row, n, vec);
      else if (state)
        r = ld_pack<T, V>(state + (t + a.W - 1) * srow, n, vec);
      st_pack<T, V>(so + j * srow, n, vec, r);
    }
  }
}

// Backward.  dv_t = dy_t silu'(v_t) with v_t formed again from the window; token t - (KW-1)'s
// dx is complete once dv_t is known.  A CTA is 8 warps along time and 32 lanes along
// channels; the filter's gradients are summed in registers, then over the CTA's warps,
// and leave as one row of partial sums per CTA.  Inputs arrive by asynchronous copies into slots of
// the thread's own, kAhead groups of KW tokens ahead: with up to 4 taps two CTAs run per SM (the
// window, the filter and its sums take 128 registers), one with more, and 80 KB or more per SM
// are on their way.
template <typename T, int KW>
constexpr int ahead_of() {
  const int group = 2 * KW * 32 * kWarpsBwd * kVecBwd * (int)sizeof(T), fit = (80 << 10) / group - 1;
  return fit >= 7 ? 7 : fit >= 3 ? 3 : 1;  // a ring of 8, 4 or 2
}
template <typename T, int KW>
constexpr int kAhead = ahead_of<T, KW>();
template <typename T, int KW, int V>
constexpr int bwd_slot_bytes() { return (kAhead<T, KW> + 1) * 2 * KW * 32 * kWarpsBwd * Pack<T, V>::BYTES; }
template <int KW, int V>
constexpr int bwd_red_bytes() { return 4 * kWarpsBwd * (KW + 1) * V * 33; }

template <typename T, int KW, int V>
__global__ void __launch_bounds__(32 * kWarpsBwd, KW <= 4 ? 2 : 1)
    short_conv_bwd_kernel(s4_short_conv_bwd_args a, bool vec, float* part, St st) {
  record_gen(st);
  extern __shared__ __align__(16) char conv_smem[];
  float(*red)[(KW + 1) * V][33] = reinterpret_cast<float(*)[(KW + 1) * V][33]>(conv_smem);
  constexpr int AHEAD = kAhead<T, KW>;
  // slots [AHEAD + 1][x, dy][KW][threads]; the sums over the CTA come after the last use of them
  Pack<T, V>* slots = reinterpret_cast<Pack<T, V>*>(conv_smem) + threadIdx.x;
  const int b = blockIdx.z, lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const Seq q = seq_of(a.lengths, nullptr, b, a.L, 0, st);
  const int h = (blockIdx.x * 32 + lane) * V, n = min(V, a.H - h);
  const int seg = blockIdx.y * kWarpsBwd + wid, t0 = seg * kSegBwd;
  float2 acc[KW + 1][V / 2];
#pragma unroll
  for (int k = 0; k <= KW; ++k)
#pragma unroll
    for (int i = 0; i < V / 2; ++i) acc[k][i] = make_float2(0.f, 0.f);

  if (n > 0 && t0 < a.L) {
    const int t1 = min(a.L, t0 + kSegBwd);
    const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
    const T* dy = static_cast<const T*>(a.dy.p) + b * a.dy.batch + h;
    T* dx = static_cast<T*>(a.dx.p) + b * a.dx.batch + h;
    const long long sb = (long long)b * (a.W - 1) * a.H + h;
    const T* state = a.state0 ? static_cast<const T*>(a.state0) + sb : nullptr;
    const T* dst = a.dstate ? static_cast<const T*>(a.dstate) + sb : nullptr;
    T* dst0 = a.dstate0 ? static_cast<T*>(a.dstate0) + sb : nullptr;
    float2 w[KW][V / 2], bias[V / 2], win[KW][V / 2], dv[KW][V / 2];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      (i % 2 ? bias[i / 2].y : bias[i / 2].x) = a.bias && i < n ? rd(a.bias + h + i) : 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k)
        (i % 2 ? w[k][i / 2].y : w[k][i / 2].x) = i < n ? rd(a.w + (long long)(h + i) * KW + k) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < KW; ++k) {
      const int t = t0 - (KW - 1) + k;
      Pack<T, V> r;
      r.zero();
      if (k < KW - 1 && t >= 0 && t < q.len)
        r = ld_pack<T, V>(x + t * a.x.row, n, vec);
      else if (k < KW - 1 && t < 0 && t >= -(a.W - 1) && state)
        r = ld_pack<T, V>(state + (t + a.W - 1) * (long long)a.H, n, vec);
      to_pairs<T, V>(r, win[k]);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) dv[k][i] = make_float2(0.f, 0.f);
    }
    // dv of the token whose input is `xi`, into the ring's place u
    const auto gradient = [&](int u, const Pack<T, V>& xi, const Pack<T, V>& di) {
      to_pairs<T, V>(xi, win[(KW - 1 + u) % KW]);
      float2 d[V / 2];
      to_pairs<T, V>(di, d);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        if (a.silu) {
          float2 v = bias[i];
#pragma unroll
          for (int k = 0; k < KW; ++k) v = fma2(w[k][i], win[(k + u) % KW][i], v);
          d[i] = mul2(d[i], silu_grad(v));
        }
        dv[(KW - 1 + u) % KW][i] = d[i];
      }
    };
    const auto add_filter = [&](int u) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        const float2 d = dv[(KW - 1 + u) % KW][i];
#pragma unroll
        for (int k = 0; k < KW; ++k) acc[k][i] = fma2(d, win[(k + u) % KW][i], acc[k][i]);
        acc[KW][i] = add2(acc[KW][i], d);
      }
    };
    // dx of the ring's oldest token (entry (k + u) % KW is k tokens after it)
    const auto input = [&](int u, float2 (&g)[V / 2]) {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        g[i] = mul2(w[KW - 1][i], dv[u % KW][i]);
#pragma unroll
        for (int k = 1; k < KW; ++k) g[i] = fma2(w[KW - 1 - k][i], dv[(k + u) % KW][i], g[i]);
      }
    };
    // token t of the loop: dv_t, and dx of token t - (KW - 1)
    const int tend = min(t1 + KW - 1, q.len);
    const bool whole = vec && n >= V;
    const auto slot = [&](int g, int which, int u) -> Pack<T, V>& {
      return slots[((g % (AHEAD + 1) * 2 + which) * KW + u) * 32 * kWarpsBwd];
    };
    const auto fetch = [&](int g) {
#pragma unroll
      for (int u = 0; u < KW; ++u) {
        const int t = t0 + g * KW + u;
        if (t >= tend) continue;
        if (whole) {
          fetch_whole<T, V>(&slot(g, 0, u), x + t * a.x.row);
          fetch_whole<T, V>(&slot(g, 1, u), dy + t * a.dy.row);
        } else {
          slot(g, 0, u) = ld_pack<T, V>(x + t * a.x.row, n, vec);
          slot(g, 1, u) = ld_pack<T, V>(dy + t * a.dy.row, n, vec);
        }
      }
      fetch_commit();
    };
#pragma unroll
    for (int g = 0; g < AHEAD; ++g) fetch(g);
    for (int tb = t0; tb < t1 + KW - 1; tb += KW) {
      const int gr = (tb - t0) / KW;
      fetch(gr + AHEAD);
      fetched_but<AHEAD>();
      // a group inside the segment, of real tokens, away from the state on return (only for whole
      // packs: rows that are not aligned took 189 us instead of 146 this way, 8 x 4095 x 1025)
      if (whole && tb > t0 && tb + KW <= min(t1, q.len) && (!dst || tb < q.len - (a.W - 1))) {
#pragma unroll
        for (int u = 0; u < KW; ++u) {
          gradient(u, slot(gr, 0, u), slot(gr, 1, u));
          add_filter(u);
          float2 g[V / 2];
          input(u, g);
          st_pairs<T, V>(dx + (tb + u - (KW - 1)) * a.dx.row, V, true, g);
        }
        continue;
      }
#pragma unroll
      for (int u = 0; u < KW; ++u) {
        const int t = tb + u;
        if (t >= t1 + KW - 1) break;
        if (t < q.len) {
          gradient(u, slot(gr, 0, u), slot(gr, 1, u));
          if (t < t1) add_filter(u);
        } else {
#pragma unroll
          for (int i = 0; i < V / 2; ++i) dv[(KW - 1 + u) % KW][i] = make_float2(0.f, 0.f);
        }
        const int tx = t - (KW - 1);
        const bool before = tx < 0;  // an input of the state on entry
        if (before ? (seg != 0 || tx < -(a.W - 1) || !dst0) : tx < t0) continue;
        float2 g[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) g[i] = make_float2(0.f, 0.f);
        if (tx < q.len) {
          input(u, g);
          const int j = tx - q.len + a.W - 1;  // its row of the state on return
          if (dst && j >= 0) {
            float2 e[V / 2];
            to_pairs<T, V>(ld_pack<T, V>(dst + j * (long long)a.H, n, vec), e);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) g[i] = add2(g[i], e[i]);
          }
        }
        if (before)
          st_pairs<T, V>(dst0 + (tx + a.W - 1) * (long long)a.H, n, vec, g);
        else
          st_pairs<T, V>(dx + tx * a.dx.row, n, vec, g);
      }
    }
  }
  fetched();
  __syncthreads();  // the slots become the sums
#pragma unroll
  for (int k = 0; k <= KW; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) red[wid][k * V + i][lane] = i % 2 ? acc[k][i / 2].y : acc[k][i / 2].x;
  __syncthreads();
  // partial sums of this CTA: part[row][k][h], k < W the taps, k = W the bias
  float* out = part + ((long long)b * gridDim.y + blockIdx.y) * (a.W + 1) * a.H;
  for (int c = threadIdx.x; c < (KW + 1) * 32 * V; c += 32 * kWarpsBwd) {
    const int k = c / (32 * V), hl = c % (32 * V), hh = blockIdx.x * 32 * V + hl;
    if (hh >= a.H) continue;
    float t = 0.f;
#pragma unroll
    for (int v = 0; v < kWarpsBwd; ++v) t += red[v][k * V + hl % V][hl / V];
    wr(out + (long long)k * a.H + hh, t);
  }
}

__global__ void __launch_bounds__(256) short_conv_sums_kernel(const float* part, int rows, int H, int W, float* dw,
                                                              float* dbias) {
  column_sums(part, rows, (long long)(W + 1) * H, (long long)(W + 1) * H, [=](long long c, float v) {
    const long long k = c / H, h = c % H;
    if (k < W)
      wr(dw + h * W + k, v);
    else if (dbias)
      wr(dbias + h, v);
  });
}

// A filter's taps are compiled in: what a longer window would multiply by 0 may be infinite.
template <typename F>
void with_taps(int W, F f) {
  switch (W) {
    case 2: return f(std::integral_constant<int, 2>{});
    case 3: return f(std::integral_constant<int, 3>{});
    case 4: return f(std::integral_constant<int, 4>{});
    case 5: return f(std::integral_constant<int, 5>{});
    case 6: return f(std::integral_constant<int, 6>{});
    case 7: return f(std::integral_constant<int, 7>{});
    default: return f(std::integral_constant<int, 8>{});
  }
}

template <typename T, int V>
cudaError_t fwd_t(const s4_short_conv_args& a, St st, cudaStream_t s) {
  const int e = sizeof(T), bytes = sizeof(Pack<T, V>);
  const bool vec = vec_ok(a.x.p, e, bytes, a.x.batch, a.x.row) && vec_ok(a.y.p, e, bytes, a.y.batch, a.y.row) &&
                   vec_ok(a.state, e, bytes, a.H) && vec_ok(a.state_out, e, bytes, a.H);
  const long long n = (long long)((a.H + V - 1) / V) * ((a.L + kSegFwd - 1) / kSegFwd);
  const dim3 grid((unsigned)((n + kThreads - 1) / kThreads), a.batch);
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.in_rows(a.x, e, a.batch, a.L, a.H);
  x.out_rows(a.y, e, a.batch, a.L, a.H);
  x.in(a.w, 4, a.W, a.H);
  x.in(a.bias, 4, a.H);
  x.in(a.lengths, 4, a.batch);
  x.in(a.index, 4, a.batch);
  x.in(a.state, e, a.H, (long long)a.slots * (a.W - 1));
  x.out(a.state_out, e, a.H, (long long)a.slots * (a.W - 1));
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  s4impl::TimedLaunch tl("short_conv", s);
  with_taps(a.W, [&](auto taps) { short_conv_kernel<T, decltype(taps)::value, V><<<grid, kThreads, 0, s>>>(a, vec, st); });
  return cudaGetLastError();
}

dim3 bwd_grid(int batch, int L, int H) {
  return dim3((H + 127) / 128, (L + kSegBwd * kWarpsBwd - 1) / (kSegBwd * kWarpsBwd), batch);
}

template <typename T>
cudaError_t bwd_t(const s4_short_conv_bwd_args& a, St st, cudaStream_t s) {
  constexpr int V = kVecBwd;
  const int e = sizeof(T), bytes = sizeof(Pack<T, V>);
  const bool vec = vec_ok(a.x.p, e, bytes, a.x.batch, a.x.row) && vec_ok(a.dy.p, e, bytes, a.dy.batch, a.dy.row) &&
                   vec_ok(a.dx.p, e, bytes, a.dx.batch, a.dx.row) && vec_ok(a.state0, e, bytes, a.H) &&
                   vec_ok(a.dstate, e, bytes, a.H) && vec_ok(a.dstate0, e, bytes, a.H);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + s4impl::kStatusBytes);
  const dim3 grid = bwd_grid(a.batch, a.L, a.H);
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.in_rows(a.x, e, a.batch, a.L, a.H);
  x.in_rows(a.dy, e, a.batch, a.L, a.H);
  x.out_rows(a.dx, e, a.batch, a.L, a.H);
  x.in(a.w, 4, a.W, a.H);
  x.in(a.bias, 4, a.H);
  x.in(a.lengths, 4, a.batch);
  for (const void* p : {a.state0, a.dstate}) x.in(p, e, a.H, (long long)a.batch * (a.W - 1));
  x.out(a.dstate0, e, a.H, (long long)a.batch * (a.W - 1));
  x.out(a.dw, 4, a.W, a.H);
  x.out(a.dbias, 4, a.H);
  x.scratch(part, 4, a.H, (long long)grid.y * grid.z * (a.W + 1));
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  {
    s4impl::TimedLaunch tl("short_conv_bwd", s);
    with_taps(a.W, [&](auto taps) {
      constexpr int KW = decltype(taps)::value, slots = bwd_slot_bytes<T, KW, V>(), sums = bwd_red_bytes<KW, V>();
      constexpr int bytes = slots > sums ? slots : sums;
      constexpr auto kernel = short_conv_bwd_kernel<T, KW, V>;
      allow_shared<kernel>(bytes);
      kernel<<<grid, 32 * kWarpsBwd, bytes, s>>>(a, vec, part, st);
    });
  }
  s4impl::TimedLaunch tl("short_conv_bwd", s);
  const long long cols = (long long)(a.W + 1) * a.H;
  short_conv_sums_kernel<<<(unsigned)((cols + 31) / 32), 256, 0, s>>>(part, (int)(grid.y * grid.z), a.H, a.W, a.dw,
                                                                     a.dbias);
  return cudaGetLastError();
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_short_conv)
#endif

cudaError_t launch_short_conv(const s4_short_conv_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return fwd_t<float, 4>(a, st, s);
  if (a.dtype == S4_BF16) return fwd_t<__nv_bfloat16, 4>(a, st, s);
  return fwd_t<__half, 4>(a, st, s);
}

size_t short_conv_bwd_scratch(int batch, int L, int H, int W) {
  const dim3 g = bwd_grid(batch, L, H);
  return sizeof(float) * (size_t)g.y * g.z * (W + 1) * H;
}

cudaError_t launch_short_conv_bwd(const s4_short_conv_bwd_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float>(a, st, s);
  if (a.dtype == S4_BF16) return bwd_t<__nv_bfloat16>(a, st, s);
  return bwd_t<__half>(a, st, s);
}

}  // namespace s4impl
