// Layer norm over rows of H channels, forward and backward:
//
//   u = (x - mean) r,  r = rsqrt(mean (x - mean)^2 + eps),  y = u w + b
//   dx = r (d - mean d - u mean(d u)),  d = dy w,  dw = sum dy u,  db = sum dy
//
// About 10 (20) operations per channel on 4 (6) bytes of 16-bit data: the bound is memory.  A row
// stays in the registers of its group of lanes (4 to 32 of a warp, or a CTA) from its read to its
// results, so every array is passed over once; the variance is formed from the centred values,
// which costs a second round of reductions and keeps its digits where the mean is large.
//
// Measured: forward 37 us on 16001 rows of 2560 channels in float16 (4.4 TB/s; a plain copy of as much takes 33), backward 51
// on 16384 rows of 2048 in bfloat16 (3.9 TB/s, 7 us of them the partial sums), 262144 rows of 128 27 and 48.  Rows whose packs
// are not whole or not aligned go element by element (16384 x 2047: 132 and 127 us); gradients of more than 8192 channels
// spill 164 to 224 bytes a thread.
#include "norm_rows.cuh"
#include "s4_sequence.h"

namespace {
using namespace s4blk;

// K sums over a group: `width` lanes of a warp, or the CTA.  Every lane of the warp takes part.
template <int MAX, int K, int KR>
__device__ __forceinline__ void row_sums(float (&v)[K], int width, float (&red)[2][KR][32], int& phase) {
  if constexpr (MAX > 128) {
    group_sums<MAX, K>(v, red, phase);
  } else {
    for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  }
}

// Pairs beyond a row's channels (of a pack with n of them) to zero.
template <int V>
__device__ __forceinline__ void cut(float2 (&v)[V / 2], int n) {
#pragma unroll
  for (int j = 0; j < V / 2; ++j) {
    if (2 * j >= n) v[j].x = 0.f;
    if (2 * j + 1 >= n) v[j].y = 0.f;
  }
}

// How threads share rows: groups of `width` lanes, `per` of them in a CTA.
struct Place {
  int lane, sub, width, per;
};
template <int MAX>
__device__ __forceinline__ Place place_of(int width) {
  if (MAX > 128) return {(int)threadIdx.x, 0, (int)blockDim.x, 1};
  return {(int)threadIdx.x & (width - 1), (int)threadIdx.x / width, width, (int)blockDim.x / width};
}

// Q rows of a group go through the rounds together, which takes half as many barriers for Q = 2, and as many more are on
// their way (two sets in all: three and four measured the same forward and 5 to 10 % slower backward).
constexpr int kSets = 2;
template <typename T, int V, int NV, int MAX, bool AHEAD, int Q>
__global__ void __launch_bounds__(MAX, NV == 1 ? 1024 / MAX : 1) layer_norm_kernel(s4_layer_norm_args a, bool vec, int lanes) {
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) char norm_smem[];
  int phase = 0, stage = 0;
  const Place p = place_of<MAX>(lanes);
  const long long step = (long long)gridDim.x * p.per;
  const float inv = 1.f / (float)a.H;
  Rows<T, T, V, NV, Q, 0, AHEAD, kSets> rows(norm_smem);
  const auto fetch = [&](long long row, int stage) {
#pragma unroll
    for (int q = 0; q < Q; ++q, row += step)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
        if (row < a.rows && c < a.H) rows.fetch_t(stage, q, i, static_cast<const T*>(a.x) + row * a.x_row + c);
      }
    fetch_commit();
  };
  // one pack of parameters per thread stays in registers
  float2 w[V / 2], b[V / 2];
  const auto ld_params = [&](int i) {
    const int c = (p.lane + i * p.width) * V;
    if (c >= a.H) return;
    ld_param<V>(w, a.w, c, a.H - c, vec, 1.f);
    ld_param<V>(b, a.b, c, a.H - c, vec, 0.f);
  };
  // every lane of a warp stays for as long as one of its groups has a row
  const long long first = (long long)blockIdx.x * p.per;
  if (AHEAD)
    for (int s = 0; s < kSets - 1; ++s) fetch(first + p.sub + s * Q * step, s);
  if (NV == 1) ld_params(0);
  for (long long at = first; at < a.rows; at += Q * step, stage = stage + 1 == kSets ? 0 : stage + 1) {
    const long long row = at + p.sub;
    if (AHEAD) {
      fetch(row + (kSets - 1) * Q * step, stage == 0 ? kSets - 1 : stage - 1);
      fetched_but<kSets - 1>();
    }
    float2 v[Q][NV][V / 2];
    float sum[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      float2 s = two(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[q][i][j] = two(0.f);
        if (row + q * step >= a.rows || c >= a.H) continue;
        rows.get_t(stage, q, i, static_cast<const T*>(a.x) + (row + q * step) * a.x_row + c, a.H - c, vec, v[q][i]);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) s = add2(s, v[q][i][j]);
      }
      sum[q] = both(s);
    }
    row_sums<MAX, Q>(sum, p.width, red, phase);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float2 mean = two(-sum[q] * inv);
      float2 s = two(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
        if (c >= a.H) continue;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[q][i][j] = add2(v[q][i][j], mean);
        if (a.H - c < V) cut<V>(v[q][i], a.H - c);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) s = fma2(v[q][i][j], v[q][i][j], s);
      }
      sum[q] = both(s);
    }
    row_sums<MAX, Q>(sum, p.width, red, phase);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float2 r = two(rsqrtf(sum[q] * inv + a.eps));
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
        if (row + q * step >= a.rows || c >= a.H) continue;
        if (NV > 1) ld_params(i);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[q][i][j] = fma2(mul2(v[q][i][j], r), w[j], b[j]);
        st_pairs<T, V>(static_cast<T*>(a.y) + (row + q * step) * a.y_row + c, a.H - c, vec, v[q][i]);
      }
    }
  }
}

// Rows of up to 4 packs a lane: a warp has R rows at once, as they lie in memory (16-bit values in 16 bits), and converts
// them in each of its three passes over them; no barriers, and the parameters are read once for R rows.
template <typename T, int V, int NV, int R>
__global__ void __launch_bounds__(128) layer_norm_warp_kernel(s4_layer_norm_args a) {
  const int lane = threadIdx.x & 31;
  const long long warp = (long long)blockIdx.x * 4 + (threadIdx.x >> 5), warps = (long long)gridDim.x * 4;
  const float inv = 1.f / (float)a.H;
  for (long long row = warp * R; row < a.rows; row += warps * R) {
    Pack<T, V> x[R][NV];
    float2 v[V / 2];
#pragma unroll
    for (int q = 0; q < R; ++q)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + 32 * i) * V;
        if (c < a.H && row + q < a.rows)
          x[q][i] = ld_whole<T, V>(static_cast<const T*>(a.x) + (row + q) * a.x_row + c);
        else
          x[q][i].zero();
      }
    float mean[R], r[R];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 s = two(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        to_pairs<T, V>(x[q][i], v);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) s = add2(s, v[j]);
      }
      mean[q] = -warp_sum(both(s)) * inv;
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float2 s = two(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if ((lane + 32 * i) * V >= a.H) continue;
        to_pairs<T, V>(x[q][i], v);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          v[j] = add2(v[j], two(mean[q]));
          s = fma2(v[j], v[j], s);
        }
      }
      r[q] = rsqrtf(warp_sum(both(s)) * inv + a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + 32 * i) * V;
      if (c >= a.H) continue;
      float2 w[V / 2], b[V / 2];
      ld_param<V>(w, a.w, c, V, true, 1.f);
      ld_param<V>(b, a.b, c, V, true, 0.f);
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (row + q >= a.rows) continue;
        to_pairs<T, V>(x[q][i], v);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[j] = fma2(mul2(add2(v[j], two(mean[q])), two(r[q])), w[j], b[j]);
        st_pairs<T, V>(static_cast<T*>(a.y) + (row + q) * a.y_row + c, V, true, v);
      }
    }
  }
}

// Two rounds of reductions per row: the sums of x and d, then those of (x - mean)^2 and d (x - mean).
// A group walks over rows with the column sums of its channels in registers; the groups of a CTA
// are summed before they leave one row of partial sums, part[CTA][2][H].
// Q rows of a group go through the rounds together, which halves the barriers of a CTA's rows.
template <typename T, int V, int NV, int MAX, bool AHEAD, int Q>
__global__ void __launch_bounds__(MAX, NV == 1 ? 512 / MAX : 1)
    layer_norm_bwd_kernel(s4_layer_norm_bwd_args a, bool vec, int lanes, float* part, St st) {
  record_gen(st);
  __shared__ float red[2][4][32];
  extern __shared__ __align__(16) char norm_smem[];
  int phase = 0, stage = 0;
  const Place p = place_of<MAX>(lanes);
  const long long step = (long long)gridDim.x * p.per;
  const float inv = 1.f / (float)a.H;
  Rows<T, T, V, NV, 2 * Q, 0, AHEAD, kSets> rows(norm_smem);
  const auto fetch = [&](long long row, int stage) {
#pragma unroll
    for (int q = 0; q < Q; ++q, row += step)
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
        if (row >= a.rows || c >= a.H) continue;
        rows.fetch_t(stage, 2 * q, i, static_cast<const T*>(a.x) + row * a.x_row + c);
        rows.fetch_t(stage, 2 * q + 1, i, static_cast<const T*>(a.dy) + row * a.dy_row + c);
      }
    fetch_commit();
  };
  float2 w[V / 2], dw[NV][V / 2], db[NV][V / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V / 2; ++j) dw[i][j] = db[i][j] = two(0.f);
  const auto ld_w = [&](int i) {
    const int c = (p.lane + i * p.width) * V;
    if (c < a.H) ld_param<V>(w, a.w, c, a.H - c, vec, 1.f);
  };
  const long long first = (long long)blockIdx.x * p.per;
  if (AHEAD)
    for (int s = 0; s < kSets - 1; ++s) fetch(first + p.sub + s * Q * step, s);
  if (NV == 1) ld_w(0);
  for (long long at = first; at < a.rows; at += Q * step, stage = stage + 1 == kSets ? 0 : stage + 1) {
    const long long row = at + p.sub;
    if (AHEAD) {
      fetch(row + (kSets - 1) * Q * step, stage == 0 ? kSets - 1 : stage - 1);
      fetched_but<kSets - 1>();
    }
    float2 v[Q][NV][V / 2], d[Q][NV][V / 2];
    float sum[2 * Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const long long at_row = row + q * step;
      float2 s0 = two(0.f), s1 = two(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[q][i][j] = d[q][i][j] = two(0.f);
        if (at_row >= a.rows || c >= a.H) continue;
        rows.get_t(stage, 2 * q, i, static_cast<const T*>(a.x) + at_row * a.x_row + c, a.H - c, vec, v[q][i]);
        rows.get_t(stage, 2 * q + 1, i, static_cast<const T*>(a.dy) + at_row * a.dy_row + c, a.H - c, vec, d[q][i]);
        if (NV > 1) ld_w(i);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          s0 = add2(s0, v[q][i][j]);
          s1 = fma2(d[q][i][j], w[j], s1);
        }
      }
      sum[2 * q] = both(s0), sum[2 * q + 1] = both(s1);
    }
    row_sums<MAX, 2 * Q>(sum, p.width, red, phase);
    float2 mean_d[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const float2 mean = two(-sum[2 * q] * inv);
      mean_d[q] = two(-sum[2 * q + 1] * inv);
      float2 s0 = two(0.f), s1 = two(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
        if (c >= a.H) continue;
        if (NV > 1) ld_w(i);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[q][i][j] = add2(v[q][i][j], mean);
        if (a.H - c < V) cut<V>(v[q][i], a.H - c);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          s0 = fma2(v[q][i][j], v[q][i][j], s0);
          s1 = fma2(mul2(d[q][i][j], w[j]), v[q][i][j], s1);
        }
      }
      sum[2 * q] = both(s0), sum[2 * q + 1] = both(s1);
    }
    row_sums<MAX, 2 * Q>(sum, p.width, red, phase);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const long long at_row = row + q * step;
      const float rs = rsqrtf(sum[2 * q] * inv + a.eps);
      const float2 r = two(rs), m = two(-rs * sum[2 * q + 1] * inv);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (p.lane + i * p.width) * V;
        if (at_row >= a.rows || c >= a.H) continue;
        if (NV > 1) ld_w(i);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 u = mul2(v[q][i][j], r);
          dw[i][j] = fma2(d[q][i][j], u, dw[i][j]);
          db[i][j] = add2(db[i][j], d[q][i][j]);
          d[q][i][j] = mul2(r, fma2(u, m, fma2(d[q][i][j], w[j], mean_d[q])));
        }
        st_pairs<T, V>(static_cast<T*>(a.dx) + at_row * a.dx_row + c, a.H - c, vec, d[q][i]);
      }
    }
  }
  if (!part) return;
  float* out = part + (long long)blockIdx.x * 2 * a.H;
  if constexpr (MAX > 128) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (p.lane + i * p.width) * V;
      if (c >= a.H) continue;
      st_pairs<float, V>(out + c, a.H - c, a.H % 4 == 0, dw[i]);
      st_pairs<float, V>(out + a.H + c, a.H - c, a.H % 4 == 0, db[i]);
    }
  } else {
    __shared__ float2 all[2][MAX][V / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        all[0][threadIdx.x][j] = dw[i][j];
        all[1][threadIdx.x][j] = db[i][j];
      }
      __syncthreads();
      const int c = (p.lane + i * p.width) * V;
      if (p.sub >= 2 || c >= a.H) continue;  // group 0 sums dw, group 1 db: there are 4 groups or more
      float2 t[V / 2];
#pragma unroll
      for (int j = 0; j < V / 2; ++j) t[j] = two(0.f);
      for (int g = 0; g < p.per; ++g)
#pragma unroll
        for (int j = 0; j < V / 2; ++j) t[j] = add2(t[j], all[p.sub][g * p.width + p.lane][j]);
      st_pairs<float, V>(out + p.sub * a.H + c, a.H - c, a.H % 4 == 0, t);
    }
  }
}

// Columns of part [rows][2][H] summed: 32 of them per CTA, a warp on every 16th row, 8 loads on their way at once.
__global__ void __launch_bounds__(512) layer_norm_sums_kernel(const float* part, int rows, int H, float* dw, float* db) {
  __shared__ float s[16][33];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + lane, pitch = 2ll * H;
  float t[8] = {};
  if (c < pitch)
    for (int r = wid; r < rows; r += 128) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (r + 16 * i < rows) t[i] += rd(part + (r + 16 * i) * pitch + c);
    }
  s[wid][lane] = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
  __syncthreads();
  if (wid != 0 || c >= pitch) return;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += s[i][lane];
  if (c < H) {
    if (dw) wr(dw + c, sum);
  } else if (db) {
    wr(db + (c - H), sum);
  }
}

// Lanes per row of a shape whose rows a warp or less holds: as few (4 at least) as hold its packs.
int lanes_for(const Shape& sh, int H, int V) {
  const int packs = (H + V - 1) / V;
  int lanes = 32;
  while (!sh.cta && sh.nv == 1 && lanes > 4 && lanes / 2 >= packs) lanes /= 2;
  return lanes;
}
// The same rows as groups for the grid's rule: `threads / per` lanes each.
template <auto Kernel>
int grid_for(long long rows, const Shape& sh, int lanes, int bytes) {
  const long long per = sh.cta ? 1 : sh.threads / lanes, warps = sh.cta ? 1 : sh.threads / 32;
  // ctas_for counts a row per warp
  return ctas_for<Kernel>((rows + per - 1) / per * warps, sh, bytes);
}

template <typename T, int V>
cudaError_t fwd_t(const s4_layer_norm_args& a, cudaStream_t s) {
  const int e = sizeof(T), b = sizeof(Pack<T, V>);
  const bool vec = vec_ok(a.x, e, b, a.x_row) && vec_ok(a.y, e, b, a.y_row) && vec_ok(a.w, 4, 16) && vec_ok(a.b, 4, 16);
  const Shape sh = shape_for(a.H, V);
  const int lanes = lanes_for(sh, a.H, V);
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.add(a.x, e, true, false, a.H, a.rows, a.x_row);
  x.add(a.y, e, false, true, a.H, a.rows, a.y_row);
  for (const float* p : {a.w, a.b}) x.in(p, 4, a.H);
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  s4impl::TimedLaunch tl("layer_norm", s);
  const int packs = (a.H + 32 * V - 1) / (32 * V);  // per lane of a warp
  // Whole rows in warps up to 4 packs a lane: 65536 rows of 512 channels in bfloat16 27 us, by CTAs 33; beyond, CTAs: 16384 rows
  // of 2048 29 us, in warps 32 to 36.
  if (vec && a.H % V == 0 && packs >= 2 && packs <= 4) {
    const auto run = [&](auto kernel, int rows) {
      const long long need = (a.rows + 4 * rows - 1) / (4 * rows), most = 16ll * s4impl::num_sms();
      kernel<<<(unsigned)(need < most ? need : most), 128, 0, s>>>(a);
      return cudaGetLastError();
    };
    // two rows a warp where that still gives every SM 16 warps
    const bool pairs = a.rows >= 32ll * s4impl::num_sms();
    if (packs <= 2) return pairs ? run(layer_norm_warp_kernel<T, V, 2, 2>, 2) : run(layer_norm_warp_kernel<T, V, 2, 1>, 1);
    return pairs ? run(layer_norm_warp_kernel<T, V, 4, 2>, 2) : run(layer_norm_warp_kernel<T, V, 4, 1>, 1);
  }
  with_shape<V>(sh, [&](auto nv, auto max) {
    constexpr int NV = decltype(nv)::value, MAX = decltype(max)::value;
    if constexpr (NV <= 2) {
      constexpr int Q = NV == 1 ? 2 : 1;
      const int bytes = NV * kRowBytes<T, T, V, Q, 0, kSets> * sh.threads;
      if (vec && a.H % V == 0 && bytes <= kMaxAhead) {
        constexpr auto kernel = layer_norm_kernel<T, V, NV, MAX, true, Q>;
        kernel<<<grid_for<kernel>(a.rows, sh, lanes, bytes), sh.threads, bytes, s>>>(a, vec, lanes);
        return;
      }
    }
    const long long per = sh.cta ? 1 : sh.threads / lanes;
    layer_norm_kernel<T, V, NV, MAX, false, 1><<<(unsigned)((a.rows + per - 1) / per), sh.threads, 0, s>>>(a, vec, lanes);
  });
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t bwd_t(const s4_layer_norm_bwd_args& a, St st, cudaStream_t s) {
  const int e = sizeof(T), b = sizeof(Pack<T, V>);
  const bool vec = vec_ok(a.x, e, b, a.x_row) && vec_ok(a.dy, e, b, a.dy_row) && vec_ok(a.dx, e, b, a.dx_row) &&
                   vec_ok(a.w, 4, 16);
  const Shape sh = shape_for(a.H, V);
  const int lanes = lanes_for(sh, a.H, V);
  int grid = 0;
  const bool sums = a.dw || a.db;
  float* part = sums ? reinterpret_cast<float*>(static_cast<char*>(a.ws) + s4impl::kStatusBytes) : nullptr;
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.add(a.x, e, true, false, a.H, a.rows, a.x_row);
  x.add(a.dy, e, true, false, a.H, a.rows, a.dy_row);
  x.add(a.dx, e, false, true, a.H, a.rows, a.dx_row);
  x.in(a.w, 4, a.H);
  for (const float* p : {a.dw, a.db}) x.out(p, 4, a.H);
  x.scratch(part, 4, a.H, (long long)(s4impl::layer_norm_bwd_scratch(a.rows, a.H) / (4ull * a.H)));
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  {
    s4impl::TimedLaunch tl("layer_norm_bwd", s);
    with_shape<V>(sh, [&](auto nv, auto max) {
      constexpr int NV = decltype(nv)::value, MAX = decltype(max)::value;
      if constexpr (NV <= 2) {
        constexpr int Q = NV == 1 ? 2 : 1;
        const int bytes = NV * kRowBytes<T, T, V, 2 * Q, 0, kSets> * sh.threads;
        if (vec && a.H % V == 0 && bytes <= kMaxAhead) {
          constexpr auto kernel = layer_norm_bwd_kernel<T, V, NV, MAX, true, Q>;
          grid = grid_for<kernel>(a.rows, sh, lanes, bytes);
          kernel<<<grid, sh.threads, bytes, s>>>(a, vec, lanes, part, st);
          return;
        }
      }
      constexpr auto kernel = layer_norm_bwd_kernel<T, V, NV, MAX, false, 1>;
      grid = grid_for<kernel>(a.rows, sh, lanes, 0);
      kernel<<<grid, sh.threads, 0, s>>>(a, vec, lanes, part, st);
    });
  }
  if (!sums) return cudaGetLastError();
  s4impl::TimedLaunch tl("layer_norm_bwd", s);
  layer_norm_sums_kernel<<<(unsigned)((2ll * a.H + 31) / 32), 512, 0, s>>>(part, grid, a.H, a.dw, a.db);
  return cudaGetLastError();
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_layer_norm)
#endif

cudaError_t launch_layer_norm(const s4_layer_norm_args& a, cudaStream_t s) {
  if (a.dtype == S4_F32) return fwd_t<float, 4>(a, s);
  return a.dtype == S4_BF16 ? fwd_t<__nv_bfloat16, 8>(a, s) : fwd_t<__half, 8>(a, s);
}

size_t layer_norm_bwd_scratch(long long rows, int H) {
  // the larger of the two pack widths' grids (of rows held by a warp each, which is the most)
  size_t most = 0;
  for (int V : {4, 8}) {
    const size_t r = (size_t)most_ctas(rows, shape_for(H, V), 16);
    most = r > most ? r : most;
  }
  return sizeof(float) * 2 * most * (size_t)H;
}

cudaError_t launch_layer_norm_bwd(const s4_layer_norm_bwd_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float, 4>(a, st, s);
  return a.dtype == S4_BF16 ? bwd_t<__nv_bfloat16, 8>(a, st, s) : bwd_t<__half, 8>(a, st, s);
}

}  // namespace s4impl
