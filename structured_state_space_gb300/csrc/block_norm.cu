// What joins two blocks, forward and backward: the gate and norm after a block, its residual
// scale, the residual sum and the norm before the next block.
//
//   v = o silu(gate), p = v r1 w_post, h' = h + scale p, y = h' r2 w_pre,
//   r1 = rsqrt(mean v^2 + eps), r2 = rsqrt(mean h'^2 + eps)
//
// About 20 operations per channel on 8 to 14 bytes: the bound is memory.  A row stays in the
// registers of one warp or one CTA from its read to its results, so every array is
// passed over once; both sums of squares are reductions over the group.
#include "s4_block.cuh"

namespace {
using namespace s4blk;
using s4impl::St;

constexpr int kMaxThreads = 512;  // of the CTA that holds a row

// K sums over the group that holds a row: a warp, or the CTA's warps.  `red` has a slot per warp;
// two sets of them alternate so that one barrier per round is enough.
template <bool CTA, int K>
__device__ __forceinline__ void group_sums(float (&v)[K], float (&red)[2][2][32], int& phase) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if constexpr (CTA) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5;
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[phase][k][wid] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(lane < nw ? red[phase][k][lane] : 0.f);
    phase ^= 1;
  }
}
template <bool CTA>
__device__ __forceinline__ float group_sum(float v, float (&red)[2][2][32], int& phase) {
  float s[1] = {v};
  group_sums<CTA, 1>(s, red, phase);
  return s[0];
}

// NV packs of V channels per thread, pack i at channel (lane + i * width) V.
template <typename T, typename R, int V, int NV, bool CTA>
__global__ void __launch_bounds__(CTA ? kMaxThreads : 128) block_norm_kernel(s4_block_norm_args a, bool vec) {
  __shared__ float red[2][2][32];
  int phase = 0;
  const int width = CTA ? blockDim.x : 32, lane = CTA ? threadIdx.x : threadIdx.x & 31;
  const long long row = CTA ? (long long)blockIdx.x : (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (row >= a.rows) return;  // whole groups only
  const T* o = static_cast<const T*>(a.o) + row * a.o_row;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + row * a.gate_row : nullptr;
  const R* h = a.h ? static_cast<const R*>(a.h) + row * a.h_row : nullptr;
  float v[NV][V], hv[NV][V];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * width) * V, n = a.H - c;
#pragma unroll
    for (int j = 0; j < V; ++j) v[i][j] = hv[i][j] = 0.f;
    if (n > 0 && S4_IN(c, a.H) && S4_IN(row, a.rows)) {
      ld_f<T, V>(o + c, n, vec, v[i]);
      if (h) ld_f<R, V>(h + c, n, vec, hv[i]);
      if (gate) {
        float g[V];
        ld_f<T, V>(gate + c, n, vec, g);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = j < n ? v[i][j] * silu(g[j]) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
  }
  float r1 = 1.f;
  if (a.w_post) r1 = rsqrtf(group_sum<CTA>(ss, red, phase) / (float)a.H + a.eps);
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * width) * V, n = a.H - c;
    if (n <= 0) continue;
    float w[V], sc[V];
    if (a.w_post) ld_f<float, V>(a.w_post + c, n, vec, w);
    if (a.scale) ld_f<float, V>(a.scale + c, n, vec, sc);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float p = a.w_post ? v[i][j] * r1 * w[j] : v[i][j];
      hv[i][j] = a.scale ? fmaf(sc[j], p, hv[i][j]) : hv[i][j] + p;
      ss = fmaf(hv[i][j], hv[i][j], ss);
    }
    st_f<R, V>(static_cast<R*>(a.h_out) + row * a.h_out_row + c, n, vec, hv[i]);
  }
  if (!a.w_pre) return;
  const float r2 = rsqrtf(group_sum<CTA>(ss, red, phase) / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * width) * V, n = a.H - c;
    if (n <= 0) continue;
    float w[V];
    ld_f<float, V>(a.w_pre + c, n, vec, w);
#pragma unroll
    for (int j = 0; j < V; ++j) w[j] *= hv[i][j] * r2;
    st_f<T, V>(static_cast<T*>(a.y) + row * a.y_row + c, n, vec, w);
  }
}

// Backward, with unit = v r1, unit2 = h' r2:
//   dh = dh' + r2 (dy w_pre - unit2 mean(dy w_pre unit2)),  dw_pre = sum_rows dy unit2
//   dp = scale dh,  dscale = sum_rows dh p,  dw_post = sum_rows dp unit
//   dv = r1 (dp w_post - unit mean(dp w_post unit)),  do = dv silu(gate),  dgate = dv o silu'(gate)
// Three rounds of reductions per row: the mean of v^2; with f = dy w_pre, those of h'^2 and f h', which
// give mean(f unit2) = r2 mean(f h'); and the last mean.  (dh being linear in sums that do not need
// r2, the third could go with the second, but where the two terms of dv nearly cancel that
// costs them their last digits.)  A group walks over rows with the three column sums of its channels in registers and leaves
// them as one row of partial sums.  AHEAD: the next row's reads are copied into slots of the
// thread's own meanwhile; at two CTAs per SM nothing else would be on its way during the sums
// (16384 rows of 2048 channels in bfloat16: 306 us without).
template <typename T, typename R, int V>
struct RowSlots {  // per thread, [..][blockDim.x]
  static constexpr int kBytes = 3 * Pack<T, V>::BYTES + 2 * Pack<R, V>::BYTES;
};
template <typename T, typename R, int V, int NV, bool CTA, bool AHEAD>
__global__ void __launch_bounds__(CTA ? kMaxThreads : 128)
    block_norm_bwd_kernel(s4_block_norm_bwd_args a, bool vec, float* part) {
  static_assert(!AHEAD || NV == 1, "");
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) char norm_smem[];
  int phase = 0;
  const int width = CTA ? blockDim.x : 32, lane = CTA ? threadIdx.x : threadIdx.x & 31;
  const int per = CTA ? 1 : blockDim.x >> 5;
  const long long first = (long long)blockIdx.x * per + (CTA ? 0 : threadIdx.x >> 5), step = (long long)gridDim.x * per;
  const float inv = 1.f / (float)a.H;
  const bool with_dy = a.dy && a.w_pre;
  float s_post[NV][V], s_scale[NV][V], s_pre[NV][V];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) s_post[i][j] = s_scale[i][j] = s_pre[i][j] = 0.f;

  // slots [2][o, gate, dy][threads] of T, then [2][h, dh'][threads] of R
  Pack<T, V>* st = reinterpret_cast<Pack<T, V>*>(norm_smem) + threadIdx.x;
  Pack<R, V>* sr = reinterpret_cast<Pack<R, V>*>(norm_smem + 6 * Pack<T, V>::BYTES * blockDim.x) + threadIdx.x;
  const int c0 = lane * V, n0 = a.H - c0;
  const auto fetch = [&](long long row, int stage) {
    if (row < a.rows && n0 >= V && S4_IN(row, a.rows)) {
      Pack<T, V>* t = st + stage * 3 * blockDim.x;
      Pack<R, V>* r = sr + stage * 2 * blockDim.x;
      fetch_whole<T, V>(t, static_cast<const T*>(a.o) + row * a.o_row + c0);
      if (a.gate) fetch_whole<T, V>(t + blockDim.x, static_cast<const T*>(a.gate) + row * a.gate_row + c0);
      if (with_dy) fetch_whole<T, V>(t + 2 * blockDim.x, static_cast<const T*>(a.dy) + row * a.dy_row + c0);
      if (a.h && with_dy) fetch_whole<R, V>(r, static_cast<const R*>(a.h) + row * a.h_row + c0);
      if (a.dh_out) fetch_whole<R, V>(r + blockDim.x, static_cast<const R*>(a.dh_out) + row * a.dh_out_row + c0);
    }
    fetch_commit();
  };
  if (AHEAD) fetch(first, 0);
  int stage = 0;
  for (long long row = first; row < a.rows; row += step, stage ^= 1) {
    const T* o = static_cast<const T*>(a.o) + row * a.o_row;
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + row * a.gate_row : nullptr;
    const R* h = a.h ? static_cast<const R*>(a.h) + row * a.h_row : nullptr;
    const T* dy = with_dy ? static_cast<const T*>(a.dy) + row * a.dy_row : nullptr;
    const R* dho = a.dh_out ? static_cast<const R*>(a.dh_out) + row * a.dh_out_row : nullptr;
    Pack<T, V>* t = st + stage * 3 * blockDim.x;
    Pack<R, V>* r = sr + stage * 2 * blockDim.x;
    if (AHEAD) {
      fetch(row + step, stage ^ 1);
      fetched_but<1>();
    }
    // array `which` of the row's pack i
    const auto ld_t = [&](int which, const T* p, int i, float (&v)[V]) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (AHEAD) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = t[which * blockDim.x].get(j);
      } else {
        ld_f<T, V>(p + c, n, vec, v);
      }
    };
    const auto ld_r = [&](int which, const R* p, int i, float (&v)[V]) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (AHEAD) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = r[which * blockDim.x].get(j);
      } else {
        ld_f<R, V>(p + c, n, vec, v);
      }
    };
    float v[NV][V], hv[NV][V], d[NV][V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = hv[i][j] = d[i][j] = 0.f;
      if (n <= 0 || !S4_IN(c, a.H)) continue;
      ld_t(0, o, i, v[i]);
      if (h && dy) ld_r(0, h, i, hv[i]);
      if (dy) ld_t(2, dy, i, d[i]);
      if (gate) {
        float g[V];
        ld_t(1, gate, i, g);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = j < n ? v[i][j] * silu(g[j]) : 0.f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    float r1 = 1.f;
    if (a.w_post) {
      float sum[1] = {ss};
      group_sums<CTA, 1>(sum, red, phase);
      r1 = rsqrtf(sum[0] * inv + a.eps);
    }
    // v -> unit; h'
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (n <= 0) continue;
      float w[V], sc[V], wp[V];
      if (a.w_post) ld_f<float, V>(a.w_post + c, n, vec, w);
      if (a.scale) ld_f<float, V>(a.scale + c, n, vec, sc);
      if (dy) ld_f<float, V>(a.w_pre + c, n, vec, wp);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] *= r1;
        const float p = a.w_post ? v[i][j] * w[j] : v[i][j];
        hv[i][j] = a.scale ? fmaf(sc[j], p, hv[i][j]) : hv[i][j] + p;
        if (dy) {
          sum[0] = fmaf(hv[i][j], hv[i][j], sum[0]);
          sum[1] = fmaf(d[i][j] * wp[j], hv[i][j], sum[1]);
        }
      }
    }
    float r2 = 0.f, m2 = 0.f;
    if (dy) {
      group_sums<CTA, 2>(sum, red, phase);
      r2 = rsqrtf(sum[0] * inv + a.eps);
      m2 = r2 * sum[1] * inv;
    }
    // d -> dh, then dp w_post
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (n <= 0) continue;
      float e[V], w[V], sc[V], wp[V];
      if (dho) ld_r(1, dho, i, e);
      if (dy) ld_f<float, V>(a.w_pre + c, n, vec, wp);
      if (a.w_post) ld_f<float, V>(a.w_post + c, n, vec, w);
      if (a.scale) ld_f<float, V>(a.scale + c, n, vec, sc);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float dh = 0.f;
        if (dy) {
          const float unit2 = hv[i][j] * r2;
          s_pre[i][j] = fmaf(d[i][j], unit2, s_pre[i][j]);
          dh = r2 * (d[i][j] * wp[j] - unit2 * m2);
        }
        if (dho) dh += e[j];
        e[j] = dh;
        const float p = a.w_post ? v[i][j] * w[j] : v[i][j];
        s_scale[i][j] = fmaf(dh, p, s_scale[i][j]);
        const float dp = a.scale ? dh * sc[j] : dh;
        s_post[i][j] = fmaf(dp, v[i][j], s_post[i][j]);
        d[i][j] = a.w_post ? dp * w[j] : dp;
        ss = fmaf(d[i][j], v[i][j], ss);
      }
      if (a.dh) st_f<R, V>(static_cast<R*>(a.dh) + row * a.dh_row + c, n, vec, e);
    }
    float m1 = 0.f;
    if (a.w_post) {
      float s1[1] = {ss};
      group_sums<CTA, 1>(s1, red, phase);
      m1 = s1[0] * inv;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (n <= 0) continue;
#pragma unroll
      for (int j = 0; j < V; ++j) d[i][j] = a.w_post ? r1 * (d[i][j] - v[i][j] * m1) : d[i][j];
      if (gate) {
        float g[V], ov[V];
        ld_t(1, gate, i, g);
        ld_t(0, o, i, ov);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float s = sigmoid(g[j]), q = g[j] * s;
          ov[j] *= d[i][j] * fmaf(q, 1.f - s, s);
          d[i][j] *= q;
        }
        st_f<T, V>(static_cast<T*>(a.dgate) + row * a.dgate_row + c, n, vec, ov);
      }
      st_f<T, V>(static_cast<T*>(a.do_) + row * a.do_row + c, n, vec, d[i]);
    }
  }
  // part[group][3][H]
  float* out = part + first * 3 * a.H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * width) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (c + j >= a.H) continue;
      out[c + j] = s_post[i][j];
      out[a.H + c + j] = s_scale[i][j];
      out[2 * a.H + c + j] = s_pre[i][j];
    }
  }
}

__global__ void __launch_bounds__(256) block_norm_sums_kernel(const float* part, int rows, int H, float* dw_post,
                                                              float* dscale, float* dw_pre) {
  column_sums(part, rows, 3ll * H, [=](long long c, float v) {
    float* out = c < H ? dw_post : c < 2ll * H ? dscale : dw_pre;
    if (out) out[c % H] = v;
  });
}

// A row's group: a warp up to 32 packs of channels per pack a thread holds, a CTA beyond.
struct Shape {
  bool cta;
  int nv, threads;
};
Shape shape_for(int H, int V) {
  const int packs = (H + V - 1) / V;
  if (packs <= 32) return {false, 1, 128};
  if (packs <= 64) return {false, 2, 128};
  int nv = 1;
  while (nv * kMaxThreads < packs) nv *= 2;
  return {true, nv, ((packs + nv - 1) / nv + 31) / 32 * 32};
}
// Groups that share the rows of the backward pass (each leaves one row of partial sums).
constexpr int kBwdCtas = 4;  // CTAs per SM
int bwd_ctas(long long rows, int H, int V, int sms) {
  const Shape sh = shape_for(H, V);
  const long long per = sh.cta ? 1 : sh.threads / 32;
  const long long need = (rows + per - 1) / per;
  return (int)(need < (long long)sms * kBwdCtas ? need : (long long)sms * kBwdCtas);
}

template <typename T, typename R, int V>
cudaError_t fwd_t(const s4_block_norm_args& a, cudaStream_t s) {
  const int et = sizeof(T), er = sizeof(R), bt = sizeof(Pack<T, V>), br = sizeof(Pack<R, V>);
  const bool vec = vec_ok(a.o, et, bt, a.o_row) && vec_ok(a.gate, et, bt, a.gate_row) && vec_ok(a.h, er, br, a.h_row) &&
                   vec_ok(a.h_out, er, br, a.h_out_row) && vec_ok(a.y, et, bt, a.y_row) && vec_ok(a.w_post, 4, 16) &&
                   vec_ok(a.scale, 4, 16) && vec_ok(a.w_pre, 4, 16);
  const Shape sh = shape_for(a.H, V);
  const long long per = sh.cta ? 1 : sh.threads / 32;
  const unsigned grid = (unsigned)((a.rows + per - 1) / per);
  s4impl::TimedLaunch tl("block_norm", s);
  if (!sh.cta && sh.nv == 1)
    block_norm_kernel<T, R, V, 1, false><<<grid, sh.threads, 0, s>>>(a, vec);
  else if (!sh.cta)
    block_norm_kernel<T, R, V, 2, false><<<grid, sh.threads, 0, s>>>(a, vec);
  else if (sh.nv == 1)
    block_norm_kernel<T, R, V, 1, true><<<grid, sh.threads, 0, s>>>(a, vec);
  else if (sh.nv == 2)
    block_norm_kernel<T, R, V, 2, true><<<grid, sh.threads, 0, s>>>(a, vec);
  else if (sh.nv == 4)
    block_norm_kernel<T, R, V, 4, true><<<grid, sh.threads, 0, s>>>(a, vec);
  else if constexpr (V == 4)  // 16384 channels in 32 bits
    block_norm_kernel<T, R, V, 8, true><<<grid, sh.threads, 0, s>>>(a, vec);
  return cudaGetLastError();
}

template <typename T, typename R, int V>
cudaError_t bwd_t(const s4_block_norm_bwd_args& a, cudaStream_t s) {
  const int et = sizeof(T), er = sizeof(R), bt = sizeof(Pack<T, V>), br = sizeof(Pack<R, V>);
  const bool vec = vec_ok(a.o, et, bt, a.o_row) && vec_ok(a.gate, et, bt, a.gate_row) && vec_ok(a.h, er, br, a.h_row) &&
                   vec_ok(a.dy, et, bt, a.dy_row) && vec_ok(a.dh_out, er, br, a.dh_out_row) &&
                   vec_ok(a.do_, et, bt, a.do_row) && vec_ok(a.dgate, et, bt, a.dgate_row) &&
                   vec_ok(a.dh, er, br, a.dh_row) && vec_ok(a.w_post, 4, 16) && vec_ok(a.scale, 4, 16) &&
                   vec_ok(a.w_pre, 4, 16);
  const Shape sh = shape_for(a.H, V);
  const int grid = bwd_ctas(a.rows, a.H, V, s4impl::num_sms());
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + s4impl::kStatusBytes);
  {
    s4impl::TimedLaunch tl("block_norm_bwd", s);
    const auto run = [&](auto kernel, int bytes) {
      if (bytes > 0) cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
      kernel<<<grid, sh.threads, bytes, s>>>(a, vec, part);
    };
    // rows of whole packs, read ahead; others as they come
    const int ahead = vec && a.H % V == 0 ? 2 * RowSlots<T, R, V>::kBytes * sh.threads : 0;
    if (!sh.cta && sh.nv == 1)
      ahead ? run(block_norm_bwd_kernel<T, R, V, 1, false, true>, ahead)
            : run(block_norm_bwd_kernel<T, R, V, 1, false, false>, 0);
    else if (!sh.cta)
      run(block_norm_bwd_kernel<T, R, V, 2, false, false>, 0);
    else if (sh.nv == 1)
      ahead ? run(block_norm_bwd_kernel<T, R, V, 1, true, true>, ahead)
            : run(block_norm_bwd_kernel<T, R, V, 1, true, false>, 0);
    else if (sh.nv == 2)
      run(block_norm_bwd_kernel<T, R, V, 2, true, false>, 0);
    else if (sh.nv == 4)
      run(block_norm_bwd_kernel<T, R, V, 4, true, false>, 0);
    else if constexpr (V == 4)  // 16384 channels in 32 bits
      run(block_norm_bwd_kernel<T, R, V, 8, true, false>, 0);
  }
  if (!a.dw_post && !a.dscale && !a.dw_pre) return cudaGetLastError();
  s4impl::TimedLaunch tl("block_norm_bwd", s);
  block_norm_sums_kernel<<<(unsigned)((3ll * a.H + 31) / 32), 256, 0, s>>>(
      part, grid * (sh.cta ? 1 : sh.threads / 32), a.H, a.dw_post, a.dscale, a.dw_pre);
  return cudaGetLastError();
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_block_norm)
#endif

cudaError_t launch_block_norm(const s4_block_norm_args& a, cudaStream_t s) {
  if (a.dtype == S4_F32) return fwd_t<float, float, 4>(a, s);
  if (a.dtype == S4_BF16)
    return a.res_f32 ? fwd_t<__nv_bfloat16, float, 8>(a, s) : fwd_t<__nv_bfloat16, __nv_bfloat16, 8>(a, s);
  return a.res_f32 ? fwd_t<__half, float, 8>(a, s) : fwd_t<__half, __half, 8>(a, s);
}

size_t block_norm_bwd_scratch(long long rows, int H) {
  // the larger of the two pack widths' partial rows
  size_t most = 0;
  for (int V : {4, 8}) {
    const Shape sh = shape_for(H, V);
    const size_t r = (size_t)bwd_ctas(rows, H, V, num_sms()) * (sh.cta ? 1 : sh.threads / 32);
    most = r > most ? r : most;
  }
  return sizeof(float) * 3 * most * (size_t)H;
}

cudaError_t launch_block_norm_bwd(const s4_block_norm_bwd_args& a, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float, float, 4>(a, s);
  if (a.dtype == S4_BF16)
    return a.res_f32 ? bwd_t<__nv_bfloat16, float, 8>(a, s) : bwd_t<__nv_bfloat16, __nv_bfloat16, 8>(a, s);
  return a.res_f32 ? bwd_t<__half, float, 8>(a, s) : bwd_t<__half, __half, 8>(a, s);
}

}  // namespace s4impl
