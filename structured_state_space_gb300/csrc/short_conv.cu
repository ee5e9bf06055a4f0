// The short causal convolution along time with SiLU, forward (prompts and single
// tokens) and backward.
//
//   v_t = bias + sum_{k<W} w[k] x[t-W+1+k],  y = v sigmoid(v)
//
// About 2 W + 5 operations on 4 bytes (16-bit types) moved: the bound is memory.  A thread
// owns V neighbouring channels (one access of 16 bytes) and walks a segment of the
// sequence with the last taps in registers, so that each input is read from memory once
// and W - 1 more times per segment from cache.
#include "s4_block.cuh"

namespace {
using namespace s4blk;
using s4impl::St;

// Taps are kept as KW = 4 or 8 (the first KW - W have weight 0 and are not read).
constexpr int kSegFwd = 16;   // tokens of a thread's segment, forward
constexpr int kSegBwd = 64;   // and backward
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
  const int t0 = seg * kSegFwd, t1 = min(a.L, t0 + kSegFwd), pad = KW - a.W;
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
  T* y = static_cast<T*>(a.y.p) + b * a.y.batch + h;
  const long long srow = a.H, sslot = (long long)(a.W - 1) * a.H;
  const T* state = a.state ? static_cast<const T*>(a.state) + (q.slot < 0 ? 0 : q.slot) * sslot + h : nullptr;

  float w[KW][V], bias[V], win[KW][V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool in = i < n && S4_IN(h + i, a.H);
    bias[i] = a.bias && in ? a.bias[h + i] : 0.f;
#pragma unroll
    for (int k = 0; k < KW; ++k) w[k][i] = in && k >= pad ? a.w[(long long)(h + i) * a.W + k - pad] : 0.f;
  }
  // the inputs before the segment: of the sequence, of the state, or zeros
#pragma unroll
  for (int k = 0; k < KW - 1; ++k) {
    const int t = t0 - (KW - 1) + k;
#pragma unroll
    for (int i = 0; i < V; ++i) win[k][i] = 0.f;
    if (t >= 0 && t < q.len) {
      ld_f<T, V>(x + t * a.x.row, n, vec, win[k]);
    } else if (t < 0 && t >= -(a.W - 1) && state && q.slot >= 0) {
      ld_f<T, V>(state + (t + a.W - 1) * srow, n, vec, win[k]);
    }
  }
  for (int t = t0; t < t1; t += KW) {
    Pack<T, V> in[KW];
#pragma unroll
    for (int u = 0; u < KW; ++u)
      if (t + u < min(t1, q.len) && S4_IN(t + u, a.L)) in[u] = ld_pack<T, V>(x + (t + u) * a.x.row, n, vec);
#pragma unroll
    for (int u = 0; u < KW; ++u) {
      if (t + u >= t1) break;
      float out[V];
      if (t + u < q.len) {
        // the window is a ring: the input of token t + u replaces that of t + u - KW
#pragma unroll
        for (int i = 0; i < V; ++i) win[(KW - 1 + u) % KW][i] = in[u].get(i);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          float v = bias[i];
#pragma unroll
          for (int k = 0; k < KW; ++k) v = fmaf(w[k][i], win[(k + u) % KW][i], v);
          out[i] = a.silu ? silu(v) : v;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) out[i] = 0.f;
      }
      if (S4_IN(t + u, a.L)) st_f<T, V>(y + (t + u) * a.y.row, n, vec, out);
    }
  }
  // The state after the last real token, row j being input len - (W-1) + j.  The thread
  // that read the channels' old state writes the new one (in place too: rows are taken
  // from rows at or after them, in ascending order).
  if (seg == 0 && a.state_out && q.slot >= 0) {
    T* so = static_cast<T*>(a.state_out) + q.slot * sslot + h;
    for (int j = 0; j < a.W - 1; ++j) {
      const int t = q.len - (a.W - 1) + j;
      Pack<T, V> r;
      r.zero();
      if (t >= 0)
        r = ld_pack<T, V>(x + t * a.x.row, n, vec);
      else if (state)
        r = ld_pack<T, V>(state + (t + a.W - 1) * srow, n, vec);
      if (S4_IN(q.slot, a.slots)) st_pack<T, V>(so + j * srow, n, vec, r);
    }
  }
}

// Backward.  dv_t = dy_t silu'(v_t) with v_t formed again from the window; token t - (KW-1)'s
// dx is complete once dv_t is known.  A CTA is 8 warps along time and 32 lanes along
// channels; the filter's gradients are summed in registers, then over the CTA's warps,
// and leave as one row of partial sums per CTA.  Inputs arrive by asynchronous copies into slots of
// the thread's own, kAhead groups of KW tokens ahead: at two CTAs per SM (the window, the filter
// and its sums take 115 registers; one CTA with 8 taps) that keeps 128 KB or more per SM on their way.
template <typename T, int KW>
constexpr int kAhead = sizeof(T) == 4 ? 2 : KW == 4 ? 4 : 5;
template <typename T, int KW, int V>
constexpr int bwd_slot_bytes() { return (kAhead<T, KW> + 1) * 2 * KW * 32 * kWarpsBwd * Pack<T, V>::BYTES; }
template <int KW, int V>
constexpr int bwd_red_bytes() { return 4 * kWarpsBwd * (KW + 1) * V * 33; }

template <typename T, int KW, int V>
__global__ void __launch_bounds__(32 * kWarpsBwd, KW == 4 ? 2 : 1)
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
  const int seg = blockIdx.y * kWarpsBwd + wid, t0 = seg * kSegBwd, pad = KW - a.W;
  float acc[KW + 1][V];
#pragma unroll
  for (int k = 0; k <= KW; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[k][i] = 0.f;

  if (n > 0 && t0 < a.L) {
    const int t1 = min(a.L, t0 + kSegBwd);
    const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
    const T* dy = static_cast<const T*>(a.dy.p) + b * a.dy.batch + h;
    T* dx = static_cast<T*>(a.dx.p) + b * a.dx.batch + h;
    const long long sb = (long long)b * (a.W - 1) * a.H + h;
    const T* state = a.state0 ? static_cast<const T*>(a.state0) + sb : nullptr;
    const T* dst = a.dstate ? static_cast<const T*>(a.dstate) + sb : nullptr;
    T* dst0 = a.dstate0 ? static_cast<T*>(a.dstate0) + sb : nullptr;
    float w[KW][V], bias[V], win[KW][V], dv[KW][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = a.bias && i < n ? a.bias[h + i] : 0.f;
#pragma unroll
      for (int k = 0; k < KW; ++k) w[k][i] = i < n && k >= pad ? a.w[(long long)(h + i) * a.W + k - pad] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) win[k][i] = dv[k][i] = 0.f;
#pragma unroll
    for (int k = 0; k < KW - 1; ++k) {
      const int t = t0 - (KW - 1) + k;
      if (t >= 0 && t < q.len)
        ld_f<T, V>(x + t * a.x.row, n, vec, win[k]);
      else if (t < 0 && t >= -(a.W - 1) && state)
        ld_f<T, V>(state + (t + a.W - 1) * (long long)a.H, n, vec, win[k]);
    }
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
        if (t >= tend || !S4_IN(t, a.L)) continue;
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
#pragma unroll
      for (int u = 0; u < KW; ++u) {
        const int t = tb + u;
        if (t >= t1 + KW - 1) break;
        const bool own = t < t1;
        if (t < q.len) {
          const Pack<T, V> xi = slot(gr, 0, u), di = slot(gr, 1, u);
#pragma unroll
          for (int i = 0; i < V; ++i) win[(KW - 1 + u) % KW][i] = xi.get(i);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float d = di.get(i);
            if (a.silu) {
              float v = bias[i];
#pragma unroll
              for (int k = 0; k < KW; ++k) v = fmaf(w[k][i], win[(k + u) % KW][i], v);
              d *= silu_grad(v);
            }
            dv[(KW - 1 + u) % KW][i] = d;
            if (own) {
#pragma unroll
              for (int k = 0; k < KW; ++k) acc[k][i] = fmaf(d, win[(k + u) % KW][i], acc[k][i]);
              acc[KW][i] += d;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) dv[(KW - 1 + u) % KW][i] = 0.f;
        }
        // dv of tokens t - (KW-1) .. t in ring order: entry (k + u) % KW is token t - (KW-1) + k
        const int tx = t - (KW - 1);
        const bool before = tx < 0;  // an input of the state on entry
        if (before ? (seg != 0 || tx < -(a.W - 1) || !dst0) : tx < t0) continue;
        float g[V];
#pragma unroll
        for (int i = 0; i < V; ++i) g[i] = 0.f;
        if (tx < q.len) {
#pragma unroll
          for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < KW; ++k) g[i] = fmaf(w[KW - 1 - k][i], dv[(k + u) % KW][i], g[i]);
          const int j = tx - q.len + a.W - 1;  // its row of the state on return
          if (dst && j >= 0) {
            float e[V];
            ld_f<T, V>(dst + j * (long long)a.H, n, vec, e);
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] += e[i];
          }
        }
        if (before)
          st_f<T, V>(dst0 + (tx + a.W - 1) * (long long)a.H, n, vec, g);
        else if (S4_IN(tx, a.L))
          st_f<T, V>(dx + tx * a.dx.row, n, vec, g);
      }
    }
  }
  fetched();
  __syncthreads();  // the slots become the sums
#pragma unroll
  for (int k = 0; k <= KW; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) red[wid][k * V + i][lane] = acc[k][i];
  __syncthreads();
  // partial sums of this CTA: part[row][k][h], k < W the taps, k = W the bias
  float* out = part + ((long long)b * gridDim.y + blockIdx.y) * (a.W + 1) * a.H;
  for (int c = threadIdx.x; c < (KW + 1) * 32 * V; c += 32 * kWarpsBwd) {
    const int k = c / (32 * V), hl = c % (32 * V), hh = blockIdx.x * 32 * V + hl;
    if (k < pad || hh >= a.H) continue;
    float t = 0.f;
#pragma unroll
    for (int v = 0; v < kWarpsBwd; ++v) t += red[v][k * V + hl % V][hl / V];
    out[(long long)(k - pad) * a.H + hh] = t;
  }
}

__global__ void __launch_bounds__(256) short_conv_sums_kernel(const float* part, int rows, int H, int W, float* dw,
                                                              float* dbias) {
  column_sums(part, rows, (long long)(W + 1) * H, [=](long long c, float v) {
    const long long k = c / H, h = c % H;
    if (k < W)
      dw[h * W + k] = v;
    else if (dbias)
      dbias[h] = v;
  });
}

template <typename T, int V>
cudaError_t fwd_t(const s4_short_conv_args& a, St st, cudaStream_t s) {
  const int e = sizeof(T), bytes = sizeof(Pack<T, V>);
  const bool vec = vec_ok(a.x.p, e, bytes, a.x.batch, a.x.row) && vec_ok(a.y.p, e, bytes, a.y.batch, a.y.row) &&
                   vec_ok(a.state, e, bytes, a.H) && vec_ok(a.state_out, e, bytes, a.H);
  const long long n = (long long)((a.H + V - 1) / V) * ((a.L + kSegFwd - 1) / kSegFwd);
  const dim3 grid((unsigned)((n + kThreads - 1) / kThreads), a.batch);
  s4impl::TimedLaunch tl("short_conv", s);
  if (a.W <= 4)
    short_conv_kernel<T, 4, V><<<grid, kThreads, 0, s>>>(a, vec, st);
  else
    short_conv_kernel<T, 8, V><<<grid, kThreads, 0, s>>>(a, vec, st);
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
  {
    s4impl::TimedLaunch tl("short_conv_bwd", s);
    const auto run = [&](auto kernel, int bytes) {
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      kernel<<<grid, 32 * kWarpsBwd, bytes, s>>>(a, vec, part, st);
    };
    const auto most = [](int x, int y) { return x > y ? x : y; };
    if (a.W <= 4)
      run(short_conv_bwd_kernel<T, 4, V>, most(bwd_slot_bytes<T, 4, V>(), bwd_red_bytes<4, V>()));
    else
      run(short_conv_bwd_kernel<T, 8, V>, most(bwd_slot_bytes<T, 8, V>(), bwd_red_bytes<8, V>()));
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
  if (a.dtype == S4_BF16) return fwd_t<__nv_bfloat16, 8>(a, st, s);
  return fwd_t<__half, 8>(a, st, s);
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
