// The selective state-space scan, backward.
//
// With a_t = 2^(d_t A log2 e), dyp = dy silu(z) and states s_t (formed again from the inputs):
//   g_t = C_t dyp_t + a_{t+1} g_{t+1}
//   dC_t = sum_h dyp_t s_t,  dB_t = sum_h d_t x_t g_t,  u_t = sum_n B_t g_t,  w_t = a_t g_t s_{t-1}
//   dx = d u + D dyp,  draw = (x u + sum_n A w) softplus',  dA = sum d w,  dz = dy ypre silu'(z)
//
// Per (token, channel, state) about 20 multiplications and additions, three exponentials and the
// sums of dB and dC over channels; per (token, channel) 14 bytes in 16 bits.  Arithmetic and the
// sums over lanes bound it.
//
// Three kernels.  (1) per segment of tokens, walking forward: each tile's state at its start and
// the gradient that reaches its end from later tiles, both from zero at the segment's ends;
// (2) where there are several segments, their joins; (3) per tile, independent of all others:
// states at every block of TB tokens, then backwards block by block, the block's states and
// factors again in registers.  Channels are summed over a CTA in a fixed order and leave
// as partial sums, which (4) adds up.
#include <limits.h>

#include "selective.cuh"

namespace {
using namespace s4sel;

template <int LPC_, int SPT_, int CPT_>
struct Geo {
  static constexpr int LPC = LPC_, SPT = SPT_, CPT = CPT_;
  static constexpr int NP = LPC * SPT, SLOTS = kThreads / LPC, HB = SLOTS * CPT;
  static constexpr int TC = 32, TB = 4;                // tokens of a tile, of a block in registers
  static constexpr int CELLS = TC * HB / kThreads;     // (token, channel) cells a thread stages
  static constexpr int WARPS = kThreads / 32;
  // shared memory in floats: cells [TC][HB][4] | B [TC][NP] | C [TC][NP] | block states | sums of dB, dC
  static constexpr int B0 = 4 * TC * HB, C0 = B0 + TC * NP, S0 = C0 + TC * NP;
  static constexpr int R0 = S0 + (TC / TB) * kThreads * CPT * SPT;
  static constexpr int END = R0 + WARPS * TB * 2 * NP;
  static constexpr int kSegBytes = 4 * (S0), kBytes = 4 * END;
};

struct Work {
  int tiles, seg_tiles, segs;  // tiles of TC tokens, per segment, segments
  int blocks;                  // channel blocks
  float *s_tile, *g_tile;      // [batch][tiles][H][N]: state at a tile's start, gradient at its end
  float *d_before, *d_after;   // [batch][tiles][H]: step sums from the segment's start / to its end
  float *s_seg, *g_seg;        // [batch][segs][H][N]: the segment's end values, then its start values
  float *d_seg;                // [batch][segs][H]
  float *part_h;               // [batch * tiles][H][N + 2]: dA, dD, ddt_bias
  float *part_bc;              // [blocks][batch][L][2 NP]
};

// The cells of a tile: step, x, dyp and dy silu'(z) of (token, channel), zeros beyond the
// sequence; softplus and gate are evaluated here, once.
template <typename T, typename G>
__device__ __forceinline__ void stage_cells(float4* cells, const s4_selective_bwd_args& a, const Chan& c, int b, int tb,
                                            int len, bool vec) {
  constexpr int HB = G::HB;
  constexpr int V0 = 16 / (int)sizeof(T), V1 = V0 < HB ? V0 : HB, V = V1 < G::CELLS ? V1 : G::CELLS;
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch;
  const T* dt = static_cast<const T*>(a.dt.p) + b * a.dt.batch;
  const T* z = a.z.p ? static_cast<const T*>(a.z.p) + b * a.z.batch : nullptr;
  const T* dy = static_cast<const T*>(a.dy.p) + b * a.dy.batch;
#pragma unroll
  for (int k = 0; k < G::CELLS / V; ++k) {
    const int cell = (k * kThreads + threadIdx.x) * V, t = tb + cell / HB, hl = cell % HB, h = c.h0 + hl;
    const int n = c.hend - h;
    if (t < len && n > 0 && S4_IN(t, a.L) && S4_IN(h, a.H)) {
      float xv[V], dv[V], zv[V], gv[V];
      ld_f<T, V>(x + t * a.x.row + h, n, vec, xv);
      ld_f<T, V>(dt + t * a.dt.row + h, n, vec, dv);
      ld_f<T, V>(dy + t * a.dy.row + h, n, vec, gv);
      if (z) ld_f<T, V>(z + t * a.z.row + h, n, vec, zv);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float d = dv[i], dyp = gv[i], dzf = 0.f;
        if (a.dt_bias && i < n) d += a.dt_bias[h + i];
        if (a.softplus) d = softplus(d);
        if (z) {
          dzf = gv[i] * silu_grad(zv[i]);
          dyp = gv[i] * silu(zv[i]);
        }
        cells[cell + i] = i < n ? make_float4(d, xv[i], dyp, dzf) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) cells[cell + i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
}

// (1) A segment's tiles in order: the state at each tile's start (from zero at the segment's
// start), and each tile's own contribution to the gradient at its start,
// R = sum_t (prod_{j<=t} a_j) C_t dyp_t; then backwards over the tiles the gradient
// that reaches each tile's end from the segment's later tiles.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) selective_ends_kernel(s4_selective_bwd_args a, Work w, bool vec, St st) {
  constexpr int LPC = G::LPC, SPT = G::SPT, CPT = G::CPT, NP = G::NP, HB = G::HB, TC = G::TC;
  extern __shared__ __align__(16) float smem[];
  float4* cells = reinterpret_cast<float4*>(smem);
  float(*sb)[NP] = reinterpret_cast<float(*)[NP]>(smem + G::B0);
  float(*sc)[NP] = reinterpret_cast<float(*)[NP]>(smem + G::C0);
  record_gen(st);
  const int b = blockIdx.z, seg = blockIdx.y;
  const Chan c = chan_of<HB>(blockIdx.x, a.H / a.G);
  const Seq q = seq_of(a.lengths, nullptr, b, a.L, 0, st);
  const int lane = threadIdx.x % LPC, slot = threadIdx.x / LPC, n0 = lane * SPT;
  const T* B = static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group;
  const T* C = static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group;
  const int first = seg * w.seg_tiles, last = min(w.tiles, first + w.seg_tiles);
  float A[CPT][SPT], s[CPT][SPT], sum[CPT];
  bool in[CPT][SPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int h = c.h0 + slot * CPT + j;
    sum[j] = 0.f;
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
      in[j][i] = h < c.hend && n0 + i < a.N;
      A[j][i] = in[j][i] ? a.A[(long long)h * a.N + n0 + i] * kLog2e : 0.f;
      s[j][i] = 0.f;
      if (in[j][i] && seg == 0 && a.state0) s[j][i] = a.state0[((long long)b * a.H + h) * a.N + n0 + i];
    }
  }
  for (int tile = first; tile < last; ++tile) {
    const int tb = tile * TC;
    const long long row = ((long long)b * w.tiles + tile) * a.H;
    float P[CPT][SPT], R[CPT][SPT], before[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int h = c.h0 + slot * CPT + j;
      before[j] = sum[j];
#pragma unroll
      for (int i = 0; i < SPT; ++i) {
        P[j][i] = 1.f;
        R[j][i] = 0.f;
        if (in[j][i]) w.s_tile[(row + h) * a.N + n0 + i] = s[j][i];
      }
      if (lane == 0 && h < c.hend) w.d_before[row + h] = sum[j];
    }
    if (tb < q.len) {
      __syncthreads();
      stage_cells<T, G>(cells, a, c, b, tb, q.len, vec);
      stage_vectors<T, TC, NP>(&sb[0][0], B, a.B.row, tb, q.len, a.N);
      stage_vectors<T, TC, NP>(&sc[0][0], C, a.C.row, tb, q.len, a.N);
      __syncthreads();
#pragma unroll 4
      for (int t = 0; t < TC; ++t) {
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          const float4 d = cells[t * HB + slot * CPT + j];
          const float dx = d.x * d.y;
          sum[j] += d.x;
#pragma unroll
          for (int i = 0; i < SPT; ++i) {
            const float f = ex2(d.x * A[j][i]);
            s[j][i] = fmaf(f, s[j][i], dx * sb[t][n0 + i]);
            P[j][i] *= f;
            R[j][i] = fmaf(P[j][i], sc[t][n0 + i] * d.z, R[j][i]);
          }
        }
      }
    }
    // the tile's own R now, the gradient at its end below
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int h = c.h0 + slot * CPT + j;
#pragma unroll
      for (int i = 0; i < SPT; ++i)
        if (in[j][i]) w.g_tile[(row + h) * a.N + n0 + i] = R[j][i];
      if (lane == 0 && h < c.hend) w.d_after[row + h] = sum[j] - before[j];
    }
  }
  float g[CPT][SPT], after[CPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int h = c.h0 + slot * CPT + j;
    after[j] = 0.f;
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
      g[j][i] = 0.f;
      if (in[j][i] && seg == w.segs - 1 && a.dstate) g[j][i] = a.dstate[((long long)b * a.H + h) * a.N + n0 + i];
    }
  }
  __syncthreads();  // d_after, written by one lane, is read by all that share the channel
  for (int tile = last - 1; tile >= first; --tile) {
    const long long row = ((long long)b * w.tiles + tile) * a.H;
    float own[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int h = c.h0 + slot * CPT + j;
      own[j] = h < c.hend ? w.d_after[row + h] : 0.f;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int h = c.h0 + slot * CPT + j;
#pragma unroll
      for (int i = 0; i < SPT; ++i) {
        if (!in[j][i]) continue;
        float* p = w.g_tile + (row + h) * a.N + n0 + i;
        const float r = *p;
        *p = g[j][i];
        g[j][i] = fmaf(ex2(own[j] * A[j][i]), g[j][i], r);
      }
      if (lane == 0 && h < c.hend) w.d_after[row + h] = after[j];
      after[j] += own[j];
    }
  }
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int h = c.h0 + slot * CPT + j;
    const long long row = ((long long)b * w.segs + seg) * a.H;
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
      if (!in[j][i]) continue;
      if (w.segs > 1) {
        w.s_seg[(row + h) * a.N + n0 + i] = s[j][i];
        w.g_seg[(row + h) * a.N + n0 + i] = g[j][i];
      } else if (a.dstate0) {
        a.dstate0[((long long)b * a.H + h) * a.N + n0 + i] = g[j][i];
      }
    }
    if (w.segs > 1 && lane == 0 && h < c.hend) w.d_seg[row + h] = sum[j];
  }
}

// (2) Joins the segments: the correction of each segment's states at its start (its predecessors'
// end state) and of its gradients at its end.
__global__ void __launch_bounds__(256) selective_joins_kernel(s4_selective_bwd_args a, Work w) {
  const int b = blockIdx.y;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, HN = (long long)a.H * a.N;
  if (i >= HN) return;
  const int h = (int)(i / a.N);
  const float A = a.A[i] * kLog2e;
  float s = 0.f, g = 0.f;
  for (int k = 0; k < w.segs; ++k) {
    const long long row = (long long)b * w.segs + k;
    const float end = w.s_seg[row * HN + i];
    w.s_seg[row * HN + i] = s;
    s = fmaf(ex2(w.d_seg[row * a.H + h] * A), s, end);
  }
  for (int k = w.segs - 1; k >= 0; --k) {
    const long long row = (long long)b * w.segs + k;
    const float r = w.g_seg[row * HN + i];
    w.g_seg[row * HN + i] = g;
    g = fmaf(ex2(w.d_seg[row * a.H + h] * A), g, r);
  }
  if (a.dstate0) a.dstate0[(long long)b * HN + i] = g;
}

// (3) One tile's gradients.
template <typename T, typename G>
__global__ void __launch_bounds__(kThreads) selective_tile_bwd_kernel(s4_selective_bwd_args a, Work w, bool vec, St st) {
  constexpr int LPC = G::LPC, SPT = G::SPT, CPT = G::CPT, NP = G::NP, HB = G::HB, TC = G::TC, TB = G::TB;
  extern __shared__ __align__(16) float smem[];
  float4* cells = reinterpret_cast<float4*>(smem);
  float(*sb)[NP] = reinterpret_cast<float(*)[NP]>(smem + G::B0);
  float(*sc)[NP] = reinterpret_cast<float(*)[NP]>(smem + G::C0);
  float* keep = smem + G::S0;
  float(*red)[TB][2 * NP] = reinterpret_cast<float(*)[TB][2 * NP]>(smem + G::R0);
  const int b = blockIdx.y, tile = blockIdx.x / w.blocks, block = blockIdx.x % w.blocks, tb = tile * TC;
  const Chan c = chan_of<HB>(block, a.H / a.G);
  const Seq q = seq_of(a.lengths, nullptr, b, a.L, 0, st);
  const int lane = threadIdx.x % LPC, slot = threadIdx.x / LPC, n0 = lane * SPT, wid = threadIdx.x / 32;
  const int wl = threadIdx.x & 31;
  const T* B = static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group;
  const T* C = static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group;
  const long long row = ((long long)b * w.tiles + tile) * a.H;
  const int live = min(TC, q.len - tb);  // <= 0: a tile of padding

  float A[CPT][SPT], g[CPT][SPT], dA[CPT][SPT], dD[CPT], db[CPT], Dv[CPT];
  float s0[CPT][SPT];
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int h = c.h0 + slot * CPT + j;
    dD[j] = db[j] = 0.f;
    Dv[j] = a.D && h < c.hend ? a.D[h] : 0.f;
    const float before = w.segs > 1 && h < c.hend ? w.d_before[row + h] : 0.f;
    const float after = w.segs > 1 && h < c.hend ? w.d_after[row + h] : 0.f;
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
      const bool in = h < c.hend && n0 + i < a.N;
      A[j][i] = in ? a.A[(long long)h * a.N + n0 + i] * kLog2e : 0.f;
      dA[j][i] = g[j][i] = s0[j][i] = 0.f;
      if (in && live > 0) {
        s0[j][i] = w.s_tile[(row + h) * a.N + n0 + i];
        g[j][i] = w.g_tile[(row + h) * a.N + n0 + i];
        if (w.segs > 1) {
          const long long at = (((long long)b * w.segs + tile / w.seg_tiles) * a.H + h) * a.N + n0 + i;
          s0[j][i] = fmaf(ex2(before * A[j][i]), w.s_seg[at], s0[j][i]);
          g[j][i] = fmaf(ex2(after * A[j][i]), w.g_seg[at], g[j][i]);
        }
      }
    }
  }
  if (live > 0) {
    stage_cells<T, G>(cells, a, c, b, tb, q.len, vec);
    stage_vectors<T, TC, NP>(&sb[0][0], B, a.B.row, tb, q.len, a.N);
    stage_vectors<T, TC, NP>(&sc[0][0], C, a.C.row, tb, q.len, a.N);
    __syncthreads();
    // states at the start of each block
    {
      float s[CPT][SPT];
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < SPT; ++i) s[j][i] = s0[j][i];
      for (int k = 0; k < TC / TB; ++k) {
#pragma unroll
        for (int j = 0; j < CPT; ++j)
#pragma unroll
          for (int i = 0; i < SPT; ++i) keep[((k * CPT + j) * SPT + i) * kThreads + threadIdx.x] = s[j][i];
        if (k + 1 == TC / TB) break;
#pragma unroll
        for (int t = k * TB; t < k * TB + TB; ++t)
#pragma unroll
          for (int j = 0; j < CPT; ++j) {
            const float4 d = cells[t * HB + slot * CPT + j];
#pragma unroll
            for (int i = 0; i < SPT; ++i)
              s[j][i] = fmaf(ex2(d.x * A[j][i]), s[j][i], d.x * d.y * sb[t][n0 + i]);
          }
      }
    }
    for (int k = TC / TB - 1; k >= 0; --k) {
      float s[TB + 1][CPT][SPT], f[TB][CPT][SPT], vy[CPT][TB], vu[CPT][TB], vw[CPT][TB];
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < SPT; ++i) s[0][j][i] = keep[((k * CPT + j) * SPT + i) * kThreads + threadIdx.x];
#pragma unroll
      for (int u = 0; u < TB; ++u) {
        const int t = k * TB + u;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          const float4 d = cells[t * HB + slot * CPT + j];
          float y = 0.f;
#pragma unroll
          for (int i = 0; i < SPT; ++i) {
            f[u][j][i] = ex2(d.x * A[j][i]);
            s[u + 1][j][i] = fmaf(f[u][j][i], s[u][j][i], d.x * d.y * sb[t][n0 + i]);
            y = fmaf(sc[t][n0 + i], s[u + 1][j][i], y);
          }
          vy[j][u] = y;
        }
      }
#pragma unroll
      for (int u = TB - 1; u >= 0; --u) {
        const int t = k * TB + u;
        float r[2 * SPT];  // dB, dC of this thread's states, over its channels
#pragma unroll
        for (int i = 0; i < 2 * SPT; ++i) r[i] = 0.f;
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          const float4 d = cells[t * HB + slot * CPT + j];
          const float dx = d.x * d.y;
          float uu = 0.f, ww = 0.f;
#pragma unroll
          for (int i = 0; i < SPT; ++i) {
            g[j][i] = fmaf(sc[t][n0 + i], d.z, g[j][i]);
            r[i] = fmaf(dx, g[j][i], r[i]);
            r[SPT + i] = fmaf(d.z, s[u + 1][j][i], r[SPT + i]);
            uu = fmaf(sb[t][n0 + i], g[j][i], uu);
            g[j][i] *= f[u][j][i];
            const float q1 = g[j][i] * s[u][j][i];
            ww = fmaf(A[j][i], q1, ww);
            dA[j][i] = fmaf(d.x, q1, dA[j][i]);
          }
          vu[j][u] = uu;
          vw[j][u] = ww;
        }
        // over the warp's channel slots (lanes LPC, 2 LPC, ... apart)
#pragma unroll
        for (int i = 0; i < 2 * SPT; ++i) {
#pragma unroll
          for (int o = LPC; o < 32; o <<= 1) r[i] += __shfl_xor_sync(0xffffffffu, r[i], o);
        }
        if (wl < LPC) {
#pragma unroll
          for (int i = 0; i < SPT; ++i) {
            red[wid][u][n0 + i] = r[i];
            red[wid][u][NP + n0 + i] = r[SPT + i];
          }
        }
      }
      // the block's cells: each lane finishes the tokens it holds the sums of
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        sum_lanes<LPC>(vy[j], lane);
        sum_lanes<LPC>(vu[j], lane);
        sum_lanes<LPC>(vw[j], lane);
        __syncwarp();  // every lane of the channel has read the block's cells
        if (lane < 4) {
#pragma unroll
          for (int i = 0; i < kOwn<LPC>; ++i) {
            const int t = k * TB + own_token<LPC>(lane, i);
            float4& cell = cells[t * HB + slot * CPT + j];
            const float4 d = cell;
            const float sig = a.softplus ? -expm1f(-d.x) : 1.f;  // softplus' = 1 - e^-d
            const float draw = t < live ? (d.y * vu[j][i] + kLn2 * vw[j][i]) * sig : 0.f;
            dD[j] = fmaf(d.z, d.y, dD[j]);
            db[j] += draw;
            cell = make_float4(d.x * vu[j][i] + Dv[j] * d.z, draw, d.w * (vy[j][i] + Dv[j] * d.y), 0.f);
          }
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < TB * 2 * NP; i += kThreads) {
        const int u = i / (2 * NP), n = i % (2 * NP);
        float v = 0.f;
#pragma unroll
        for (int x = 0; x < G::WARPS; ++x) v += red[x][u][n];
        const int t = tb + k * TB + u;
        if (t < a.L && S4_IN(t, a.L)) w.part_bc[(((long long)block * a.batch + b) * a.L + t) * 2 * NP + n] = v;
      }
      __syncthreads();
    }
  }
  // outputs
  constexpr int V0 = 16 / (int)sizeof(T), V1 = V0 < HB ? V0 : HB, V = V1 < G::CELLS ? V1 : G::CELLS;
#pragma unroll
  for (int k = 0; k < G::CELLS / V; ++k) {
    const int cell = (k * kThreads + threadIdx.x) * V, t = tb + cell / HB, h = c.h0 + cell % HB, n = c.hend - h;
    if (t >= a.L || n <= 0 || !S4_IN(t, a.L)) continue;
    float o[3][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool on = t < q.len;
      const float4 d = on ? cells[cell + i] : make_float4(0.f, 0.f, 0.f, 0.f);
      o[0][i] = d.x;
      o[1][i] = d.y;
      o[2][i] = d.z;
    }
    st_f<T, V>(static_cast<T*>(a.dx.p) + b * a.dx.batch + t * a.dx.row + h, n, vec, o[0]);
    st_f<T, V>(static_cast<T*>(a.ddt.p) + b * a.ddt.batch + t * a.ddt.row + h, n, vec, o[1]);
    if (a.dz.p) st_f<T, V>(static_cast<T*>(a.dz.p) + b * a.dz.batch + t * a.dz.row + h, n, vec, o[2]);
  }
  if (live <= 0) {
    for (int i = threadIdx.x; i < min(TC, a.L - tb) * 2 * NP; i += kThreads)
      w.part_bc[(((long long)block * a.batch + b) * a.L + tb) * 2 * NP + i] = 0.f;
  }
  // this tile's part of dA, dD, ddt_bias
  float* ph = w.part_h + row * (a.N + 2);
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int h = c.h0 + slot * CPT + j;
#pragma unroll
    for (int o = 1; o < (LPC < 4 ? LPC : 4); o <<= 1) {
      dD[j] += __shfl_xor_sync(0xffffffffu, dD[j], o);
      db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
    }
    if (h >= c.hend) continue;
#pragma unroll
    for (int i = 0; i < SPT; ++i)
      if (n0 + i < a.N) ph[(long long)h * a.N + n0 + i] = dA[j][i];
    if (lane == 0) {
      ph[(long long)a.H * a.N + h] = dD[j];
      ph[(long long)a.H * (a.N + 1) + h] = db[j];
    }
  }
}

// (4) The partial sums: over tiles and sequences ...
__global__ void __launch_bounds__(256) selective_sums_kernel(const float* part, int rows, int H, int N, float* dA, float* dD,
                                                             float* db) {
  column_sums(part, rows, (long long)H * (N + 2), [=](long long c, float v) {
    const long long HN = (long long)H * N;
    if (c < HN)
      dA[c] = v;
    else if (c < HN + H) {
      if (dD) dD[c - HN] = v;
    } else if (db) {
      db[c - HN - H] = v;
    }
  });
}
// ... and dB, dC over a group's channel blocks.
template <typename T>
__global__ void __launch_bounds__(256) selective_vectors_kernel(s4_selective_bwd_args a, Work w, int NP, int per) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, rows = (long long)a.batch * a.L;
  const int cols = a.G * 2 * NP;
  if (i >= rows * cols) return;
  const long long row = i / cols;
  const int g = (int)(i % cols) / (2 * NP), n = (int)(i % (2 * NP));
  float v = 0.f;
  for (int k = 0; k < per; ++k) v += w.part_bc[((long long)(g * per + k) * rows + row) * 2 * NP + n];
  const int state = n % NP;
  if (state >= a.N) return;
  T* out = static_cast<T*>(n < NP ? a.dB : a.dC);
  out[(row * a.G + g) * a.N + state] = from_f<T>(v);
}

// The lanes, states per lane and channels per thread that hold N states.
template <typename F>
auto with_states(int N, F f) {
  if (N <= 4) return f(Geo<1, 4, 1>{});
  if (N <= 8) return f(Geo<2, 4, 1>{});
  if (N <= 16) return f(Geo<4, 4, 2>{});
  if (N <= 32) return f(Geo<8, 4, 2>{});
  if (N <= 64) return f(Geo<16, 4, 2>{});
  if (N <= 128) return f(Geo<32, 4, 2>{});
  return f(Geo<32, 8, 1>{});
}

constexpr int kWarps = 16;  // per SM that the first kernel's segments are meant to fill

// Sizes and the workspace's layout (pointers relative to a null base when ws is null).
template <typename G>
Work layout(int batch, int L, int H, int N, int Gr, char* ws, size_t* total) {
  Work w;
  w.tiles = (L + G::TC - 1) / G::TC;
  w.blocks = Gr * ((H / Gr + G::HB - 1) / G::HB);
  const long long ctas = (long long)batch * w.blocks, want = (long long)s4impl::num_sms() * kWarps / (kThreads / 32);
  long long segs = (want + ctas - 1) / ctas;
  if (segs > w.tiles / 4) segs = w.tiles / 4;
  if (segs < 1) segs = 1;
  w.seg_tiles = (int)((w.tiles + segs - 1) / segs);
  w.segs = (w.tiles + w.seg_tiles - 1) / w.seg_tiles;
  const size_t HN = (size_t)H * N, bt = (size_t)batch * w.tiles, bs = (size_t)batch * w.segs;
  size_t at = s4impl::kStatusBytes;
  auto take = [&](size_t n) {
    float* p = reinterpret_cast<float*>(ws + at);
    at += s4impl::align256(4 * n);
    return p;
  };
  w.s_tile = take(bt * HN);
  w.g_tile = take(bt * HN);
  w.d_before = take(bt * H);
  w.d_after = take(bt * H);
  w.s_seg = take(w.segs > 1 ? bs * HN : 0);
  w.g_seg = take(w.segs > 1 ? bs * HN : 0);
  w.d_seg = take(w.segs > 1 ? bs * H : 0);
  w.part_h = take(bt * H * (N + 2));
  w.part_bc = take((size_t)w.blocks * batch * L * 2 * G::NP);
  if (total) *total = (long long)w.blocks * w.tiles > INT_MAX ? 0 : at;  // CTAs of one launch
  return w;
}

template <typename T>
cudaError_t bwd_t(const s4_selective_bwd_args& a, St st, cudaStream_t s) {
  const int e = sizeof(T);
  const auto ok = [&](const auto& r) { return vec_ok(r.p, e, 16, r.batch, r.row); };
  const bool vec = ok(a.x) && ok(a.dt) && ok(a.z) && ok(a.dy) && ok(a.dx) && ok(a.ddt) && ok(a.dz) &&
                   (a.G == 1 || (a.H / a.G) * e % 16 == 0);
  with_states(a.N, [&](auto geo) {
    using G = decltype(geo);
    const Work w = layout<G>(a.batch, a.L, a.H, a.N, a.G, static_cast<char*>(a.ws), nullptr);
    cudaFuncSetAttribute(selective_ends_kernel<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSegBytes);
    cudaFuncSetAttribute(selective_tile_bwd_kernel<T, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kBytes);
    {
      s4impl::TimedLaunch tl("selective_bwd", s);
      selective_ends_kernel<T, G><<<dim3(w.blocks, w.segs, a.batch), kThreads, G::kSegBytes, s>>>(a, w, vec, st);
    }
    const long long HN = (long long)a.H * a.N;
    if (w.segs > 1) {
      s4impl::TimedLaunch tl("selective_bwd", s);
      selective_joins_kernel<<<dim3((unsigned)((HN + 255) / 256), a.batch), 256, 0, s>>>(a, w);
    }
    {
      s4impl::TimedLaunch tl("selective_bwd", s);
      selective_tile_bwd_kernel<T, G>
          <<<dim3((unsigned)w.blocks * w.tiles, a.batch), kThreads, G::kBytes, s>>>(a, w, vec, st);
    }
    {
      s4impl::TimedLaunch tl("selective_bwd", s);
      const long long cols = (long long)a.H * (a.N + 2);
      selective_sums_kernel<<<(unsigned)((cols + 31) / 32), 256, 0, s>>>(w.part_h, a.batch * w.tiles, a.H, a.N, a.dA, a.dD,
                                                                        a.ddt_bias);
    }
    s4impl::TimedLaunch tl("selective_bwd", s);
    const long long n = (long long)a.batch * a.L * a.G * 2 * G::NP;
    selective_vectors_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a, w, G::NP, w.blocks / a.G);
  });
  return cudaGetLastError();
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_selective_bwd)
#endif

size_t selective_bwd_bytes(int batch, int L, int H, int N, int G) {
  size_t total = 0;
  with_states(N, [&](auto geo) { layout<decltype(geo)>(batch, L, H, N, G, nullptr, &total); });
  return total;
}

cudaError_t launch_selective_bwd(const s4_selective_bwd_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float>(a, st, s);
  if (a.dtype == S4_BF16) return bwd_t<__nv_bfloat16>(a, st, s);
  return bwd_t<__half>(a, st, s);
}

}  // namespace s4impl
