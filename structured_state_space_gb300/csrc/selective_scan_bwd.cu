// The selective state-space scan, backward.
//
// With a_t = 2^(d_t A log2 e), dyp = dy silu(z) and states s_t (formed again from the inputs):
//   g_t = C_t dyp_t + a_{t+1} g_{t+1}
//   dC_t = sum_h dyp_t s_t,  dB_t = sum_h d_t x_t g_t,  u_t = sum_n B_t g_t,  w_t = a_t g_t s_{t-1}
//   dx = d u + D dyp,  draw = (x u + sum_n A w) softplus',  dA = sum d w,  dz = dy ypre silu'(z)
//
// Per (token, channel, state) 22 multiplications and additions, four exponentials and the sums of dB
// and dC over channels; per (token, channel) 14 bytes in 16 bits.  Instructions bound it, about 44
// clocks of an SM quarter for 32 (token, channel, state), and close behind what shared memory and the
// shuffles deliver to registers.
//
// Four kernels.  (1) per segment of tokens, walking forward: the state at each tile's start, from
// a zero start, and the gradient at the segment's start from a zero end; (2) joins the
// segments; (3) per segment, walking backward tile by tile with the gradient in registers:
// the states at every block of TB tokens, then block by block the states again, in registers,
// and the gradients.  Channels and tokens are summed in a fixed order: over a thread's channels,
// its warp, its CTA, then as partial sums, which (4) adds up.  With one segment there is no (2).
//
// Measured: 897 us on 4 sequences of 4096 tokens, 2048 channels and 16 states in bfloat16: (1) 200, (2) 20,
// (3) 650, (4) 28.  The instances spill some registers: (3) 20 bytes of stores a thread with 16 states in 16 bits,
// up to 48 with other numbers, and 590 to 720 with more than 128 states.
#include <limits.h>

#include "selective.cuh"

namespace {
using namespace s4sel;

template <int LPC_, int SPT_>
struct Geo {
  static constexpr int LPC = LPC_, SPT = SPT_, NP = LPC * SPT, CPT = 2, SLOTS = 32 / LPC;
  static constexpr int CH = SLOTS * CPT;                 // channels of a warp
  static constexpr int WARPS = kThreads / 32, HB = WARPS * CH;  // and of a CTA
  static constexpr int TC = LPC == 1 ? 8 : 16, TB = 4;   // tokens of a tile, of a block in registers
  static constexpr int OWN = TC / 4 * kOwn<LPC>;         // tokens of a tile that a lane stages and finishes
  // shared memory in floats: (step, x) and (dyp, dy silu') of channel pairs, [TC][ROW] each | B, C [TC][NP] | states at
  // blocks | sums of dB, dC [2][WARPS][TB][RROW]
  static constexpr int ROW = WARPS * SLOTS * 4 + row_pad(LPC, WARPS * SLOTS * 4), RROW = 2 * NP + 16;
  static constexpr int B0 = 2 * TC * ROW, C0 = B0 + TC * NP, S0 = C0 + TC * NP;
  // | the tile before: x, dt, z, dy [4][OWN][kThreads] packs of 2 | B, C | its states
  static constexpr int VECS = TC * NP / kThreads > 0 ? TC * NP / kThreads : 1;  // elements of B, of C a thread stages
  static constexpr int R0 = S0 + TC / TB * kThreads * CPT * SPT, X0 = R0 + 2 * WARPS * TB * RROW;
  template <typename T>
  static constexpr int V0() { return X0 + 4 * OWN * kThreads * 2 * (int)sizeof(T) / 4; }
  template <typename T>
  static constexpr int N0() { return V0<T>() + 2 * VECS * kThreads * (int)sizeof(T) / 4; }
  template <typename T>
  static constexpr int kBytes() { return 4 * (N0<T>() + kThreads * CPT * SPT); }
  static constexpr int GT = 16 / SPT;                    // tokens whose sums over channels are formed together
};
// (1): a warp's tile of TT tokens: (step, step x) [TT][DROW] and dyp [TT][PROW] of channel pairs | B, C
// [TT][NP]
template <int LPC_, int SPT_, int TC_>
struct EndsGeo {
  static constexpr int LPC = LPC_, SPT = SPT_, NP = LPC * SPT, CPT = 2, SLOTS = 32 / LPC, CH = SLOTS * CPT;
  static constexpr int TT = LPC == 1 || NP > 64 ? 4 : 8, TC = TC_;  // its tile, and (3)'s
  static constexpr int OWN = TT / 4 * kOwn<LPC>;
  // | the next tile's x, dt, z, dy [4][OWN][32] packs of 2 | its B, C
  static constexpr int DROW = SLOTS * 4 + row_pad(LPC, SLOTS * 4), PROW = SLOTS * 2 + row_pad(LPC, SLOTS * 2);
  static constexpr int P0 = TT * DROW, B0 = P0 + TT * PROW, C0 = B0 + TT * NP, X0 = C0 + TT * NP;
  static constexpr int V0 = X0 + 4 * OWN * 32 * 2, END = V0 + 2 * TT * NP, kBytes = 4 * END * (kThreads / 32);
  static constexpr int VECS = TT * NP / 32;              // elements of B, of C that a lane stages
};

struct Work {
  int tiles, seg_tiles, segs;  // tiles of TC tokens, per segment, segments
  int blocks;                  // CTAs over the channels
  float *s_tile, *d_before;    // [batch][tiles][H][N], [batch][tiles][H]: state and step sum at a tile's start
  float *s_seg, *g_seg;        // [batch][segs][H][N]: a segment's ends from zero, then its corrections
  float *d_seg;                // [batch][segs][H]
  float *part_h;               // [batch * segs][pitch_h]: dA [H][N], dD [H], ddt_bias [H]
  long long pitch_h;           // H (N + 2) rounded up to whole words of 16 bytes, which dA is stored in
  float *part_bc;              // [blocks][batch][L][2 NP]
};

// What a lane reads of one token and its 2 channels.
template <typename T>
struct Cell {
  Pack<T, 2> x, dt, z, dy;
};
// A lane's slots for OWN of them in shared memory, STRIDE lanes apart: [4][OWN][STRIDE].
template <typename T, int OWN, int STRIDE>
struct Cells {
  Pack<T, 2>* s;
  __device__ __forceinline__ void fetch(int k, const s4_selective_bwd_args& a, const T* x, const T* dt, const T* z,
                                        const T* dy, long long t) {
    fetch_whole<T, 2>(s + k * STRIDE, x + t * a.x.row);
    fetch_whole<T, 2>(s + (OWN + k) * STRIDE, dt + t * a.dt.row);
    fetch_whole<T, 2>(s + (2 * OWN + k) * STRIDE, dy + t * a.dy.row);
    if (z) fetch_whole<T, 2>(s + (3 * OWN + k) * STRIDE, z + t * a.z.row);
  }
  __device__ __forceinline__ void load(int k, const s4_selective_bwd_args& a, const T* x, const T* dt, const T* z,
                                       const T* dy, long long t, int n, bool vec) {
    s[k * STRIDE] = ld_pack<T, 2>(x + t * a.x.row, n, vec);
    s[(OWN + k) * STRIDE] = ld_pack<T, 2>(dt + t * a.dt.row, n, vec);
    s[(2 * OWN + k) * STRIDE] = ld_pack<T, 2>(dy + t * a.dy.row, n, vec);
    if (z) s[(3 * OWN + k) * STRIDE] = ld_pack<T, 2>(z + t * a.z.row, n, vec);
  }
  __device__ __forceinline__ Cell<T> get(int k, const T* z) const {
    Cell<T> c;
    c.x = s[k * STRIDE];
    c.dt = s[(OWN + k) * STRIDE];
    c.dy = s[(2 * OWN + k) * STRIDE];
    if (z) c.z = s[(3 * OWN + k) * STRIDE];
    return c;
  }
};
// Step sizes, inputs, dyp and dy silu'(z) of a cell.
template <typename T>
__device__ __forceinline__ void eval_cell(const Cell<T>& c, bool gate, bool soft, float2 bias, float2& d, float2& x,
                                          float2& p, float2& zf) {
  d = add2(make_float2(c.dt.get(0), c.dt.get(1)), bias);
  if (soft) d = softplus2(d);
  x = make_float2(c.x.get(0), c.x.get(1));
  p = make_float2(c.dy.get(0), c.dy.get(1));
  zf = make_float2(0.f, 0.f);
  if (gate) {
    const float2 z = make_float2(c.z.get(0), c.z.get(1));
    const float2 s = sigmoid(z), q = mul2(z, s);  // silu = q, silu' = s + q (1 - s)
    zf = mul2(p, fma2(q, fma2(s, make_float2(-1.f, -1.f), make_float2(1.f, 1.f)), s));
    p = mul2(p, q);
  }
}

// SPT states of a channel, as pairs; the states beyond N as zeros.
template <int SPT>
__device__ __forceinline__ void ld_states(float2 (&v)[SPT / 2], const float* p, int n, bool vec) {
  float f[SPT];
  ld_f<float, SPT>(p, n, vec, f);
#pragma unroll
  for (int i = 0; i < SPT / 2; ++i) v[i] = make_float2(f[2 * i], f[2 * i + 1]);
}
template <int SPT>
__device__ __forceinline__ void st_states(float* p, int n, bool vec, const float2 (&v)[SPT / 2]) {
  float f[SPT];
#pragma unroll
  for (int i = 0; i < SPT / 2; ++i) {
    f[2 * i] = v[i].x;
    f[2 * i + 1] = v[i].y;
  }
  st_f<float, SPT>(p, n, vec, f);
}

// A warp's task and its lane's place in it.
template <typename G>
struct Place {
  int lane, slot, n0, h, nh, ns;  // lane of the channels, slot, first state, first channel, channels there are / it stages
  __device__ __forceinline__ Place(int h0, int hend) {
    const int wl = threadIdx.x & 31;
    lane = wl % G::LPC;
    slot = wl / G::LPC;
    n0 = lane * G::SPT;
    h = h0 + slot * G::CPT;
    nh = hend - h;
    ns = G::LPC > 4 && lane >= 4 ? 0 : nh;
  }
  // the k-th token of a tile that this lane owns
  __device__ __forceinline__ int token(int k) const {
    return k / kOwn<G::LPC> * 4 + own_token<G::LPC>(lane, k % kOwn<G::LPC>);
  }
};

// (1) A warp per channel block and segment, in tiles of TT tokens read ahead by one.  The gradient
// at the segment's start is R = sum_t (prod_{j<=t} a_j) C_t dyp_t.
template <typename T, typename G, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 4) selective_ends_kernel(s4_selective_bwd_args a, Work w, bool vec, bool vecbc,
                                                                     bool vecn, St st) {
  constexpr int LPC = G::LPC, SPT = G::SPT, CPT = G::CPT, NP = G::NP, CH = G::CH, TT = G::TT, OWN = G::OWN;
  constexpr int V0 = 16 / (int)sizeof(T), VB = V0 < G::VECS ? V0 : G::VECS, NB = G::VECS / VB;
  extern __shared__ __align__(16) float smem[];
  float* mine = smem + threadIdx.x / 32 * G::END;
  float4(*sd)[G::DROW / 4] = reinterpret_cast<float4(*)[G::DROW / 4]>(mine);
  float2(*sp)[G::PROW / 2] = reinterpret_cast<float2(*)[G::PROW / 2]>(mine + G::P0);
  float(*sb)[NP] = reinterpret_cast<float(*)[NP]>(mine + G::B0);
  float(*sc)[NP] = reinterpret_cast<float(*)[NP]>(mine + G::C0);
  record_gen(st);
  const int b = blockIdx.y, wl = threadIdx.x & 31, blocks = chan_blocks<CH>(a.H, a.G);
  const Seq q = seq_of(a.lengths, nullptr, b, a.L, 0, st);
  const long long task = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (task >= (long long)blocks * w.segs) return;
  const int seg = (int)(task / blocks);
  const Chan c = chan_of<CH>((int)(task % blocks), a.H / a.G);
  const Place<G> p(c.h0, c.hend);
  const int lane = p.lane, slot = p.slot, n0 = p.n0, h = p.h, nh = p.nh, nn = a.N - n0;
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
  const T* dt = static_cast<const T*>(a.dt.p) + b * a.dt.batch + h;
  const T* z = a.z.p ? static_cast<const T*>(a.z.p) + b * a.z.batch + h : nullptr;
  const T* dy = static_cast<const T*>(a.dy.p) + b * a.dy.batch + h;
  const T* B = static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group;
  const T* C = static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group;
  const int t0 = seg * w.seg_tiles * G::TC, t1 = min(a.L, t0 + w.seg_tiles * G::TC), live = min(t1, q.len);
  // this lane's slots of the next tile
  Cells<T, OWN, 32> next{reinterpret_cast<Pack<T, 2>*>(mine + G::X0) + wl};
  Pack<T, VB>* nextv = reinterpret_cast<Pack<T, VB>*>(mine + G::V0) + wl;
  const auto fetch = [&](int tb) {
    if (WHOLE && tb + TT <= live) {
#pragma unroll
      for (int k = 0; k < OWN; ++k) next.fetch(k, a, x, dt, z, dy, tb + p.token(k));
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = (k * 32 + wl) * VB, t = tb + i / NP;
        fetch_whole<T, VB>(nextv + k * 32, B + t * a.B.row + i % NP);
        fetch_whole<T, VB>(nextv + (NB + k) * 32, C + t * a.C.row + i % NP);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int t = tb + p.token(k);
      next.load(k, a, x, dt, z, dy, t, t < live ? p.ns : 0, vec);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = (k * 32 + wl) * VB, t = tb + i / NP, n = t < live ? a.N - i % NP : 0;
      nextv[k * 32] = ld_pack<T, VB>(B + t * a.B.row + i % NP, n, vecbc);
      nextv[(NB + k) * 32] = ld_pack<T, VB>(C + t * a.C.row + i % NP, n, vecbc);
    }
  };
  if (t0 < live) fetch(t0);  // before the reads below, which take as long
  float2 A[CPT][SPT / 2], s[CPT][SPT / 2], P[CPT][SPT / 2], R[CPT][SPT / 2], sum = make_float2(0.f, 0.f);
  const float2 bias = make_float2(a.dt_bias && nh > 0 ? rd(a.dt_bias + h) : 0.f, a.dt_bias && nh > 1 ? rd(a.dt_bias + h + 1) : 0.f);
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int n = j < nh ? nn : 0;
    ld_states<SPT>(A[j], a.A + (long long)(h + j) * a.N + n0, n, vecn);
    if (seg == 0 && a.state0)
      ld_states<SPT>(s[j], a.state0 + ((long long)b * a.H + h + j) * a.N + n0, n, vecn);
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) {
      A[j][i] = mul2(A[j][i], make_float2(kLog2e, kLog2e));
      if (!(seg == 0 && a.state0)) s[j][i] = make_float2(0.f, 0.f);
      P[j][i] = make_float2(1.f, 1.f);
      R[j][i] = make_float2(0.f, 0.f);
    }
  }
  for (int tb = t0; tb < t1; tb += TT) {
    if (tb % G::TC == 0) {  // a tile of (3) starts
      const long long row = ((long long)b * w.tiles + tb / G::TC) * a.H + h;
      float2 all = sum;  // over the lanes that own tokens
#pragma unroll
      for (int o = 1; o < (LPC < 4 ? LPC : 4); o <<= 1) {
        all.x += __shfl_xor_sync(0xffffffffu, all.x, o);
        all.y += __shfl_xor_sync(0xffffffffu, all.y, o);
      }
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        if (j >= nh) continue;
        st_states<SPT>(w.s_tile + (row + j) * a.N + n0, nn, vecn, s[j]);
        if (lane == 0) wr(w.d_before + row + j, j ? all.y : all.x);
      }
      if (tb >= live) continue;
    }
    if (tb >= live) continue;
    fetched();
    __syncwarp();  // the tile before has been read
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      float2 d, xv, pv, zf;
      eval_cell<T>(next.get(k, z), z != nullptr, a.softplus, bias, d, xv, pv, zf);
      const int t = p.token(k);
      if (tb + t >= live) d = make_float2(0.f, 0.f);  // padding keeps the state
      sum = add2(sum, d);
      const float2 dx = mul2(d, xv);
      if (LPC <= 4 || lane < 4) {
        sd[t][slot] = make_float4(d.x, d.y, dx.x, dx.y);
        sp[t][slot] = pv;
      }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = (k * 32 + wl) * VB;
      const Pack<T, VB> pb = nextv[k * 32], pc = nextv[(NB + k) * 32];
#pragma unroll
      for (int e = 0; e < VB; ++e) {
        (&sb[0][0])[i + e] = pb.get(e);
        (&sc[0][0])[i + e] = pc.get(e);
      }
    }
    __syncwarp();
    if (tb + TT < live) fetch(tb + TT);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float4 d = sd[t][slot];
      const float2 pv = sp[t][slot];
      const float2 dd[CPT] = {make_float2(d.x, d.x), make_float2(d.y, d.y)};
      const float2 xx[CPT] = {make_float2(d.z, d.z), make_float2(d.w, d.w)};
      const float2 pp[CPT] = {make_float2(pv.x, pv.x), make_float2(pv.y, pv.y)};
#pragma unroll
      for (int i = 0; i < SPT / 2; i += 2) {
        const float4 b4 = *reinterpret_cast<const float4*>(&sb[t][n0 + 2 * i]);
        const float4 c4 = *reinterpret_cast<const float4*>(&sc[t][n0 + 2 * i]);
        const float2 bv[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
        const float2 cv[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < CPT; ++j) {
            const float2 f = ex2(mul2(dd[j], A[j][i + e]));
            s[j][i + e] = fma2(f, s[j][i + e], mul2(xx[j], bv[e]));
            P[j][i + e] = mul2(P[j][i + e], f);
            R[j][i + e] = fma2(P[j][i + e], mul2(pp[j], cv[e]), R[j][i + e]);
          }
      }
    }
  }
#pragma unroll
  for (int o = 1; o < (LPC < 4 ? LPC : 4); o <<= 1) {
    sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
    sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
  }
  const long long row = ((long long)b * w.segs + seg) * a.H + h;
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (j >= nh) continue;
    st_states<SPT>(w.s_seg + (row + j) * a.N + n0, nn, vecn, s[j]);
    st_states<SPT>(w.g_seg + (row + j) * a.N + n0, nn, vecn, R[j]);
    if (lane == 0) wr(w.d_seg + row + j, j ? sum.y : sum.x);
  }
}

// (2) Joins the segments: what to add to each segment's states for its predecessors, times
// 2^(A steps since its start), and the gradient at its end.  A thread per state, 8 segments'
// loads under way at a time.
__global__ void __launch_bounds__(128) selective_joins_kernel(s4_selective_bwd_args a, Work w) {
  const int b = blockIdx.y;
  const long long i = (long long)blockIdx.x * 128 + threadIdx.x, HN = (long long)a.H * a.N;
  if (i >= HN) return;
  const float A = rd(a.A + i) * kLog2e;
  float* sp = w.s_seg + (long long)b * w.segs * HN + i;
  float* gp = w.g_seg + (long long)b * w.segs * HN + i;
  const float* dp = w.d_seg + (long long)b * w.segs * a.H + i / a.N;
  float s = 0.f, g = a.dstate ? rd(a.dstate + (long long)b * HN + i) : 0.f;
  for (int k0 = 0; k0 < w.segs; k0 += 8) {
    float sv[8], gv[8], ds[8], dg[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = k0 + e, r = w.segs - 1 - k;
      const bool in = k < w.segs;
      sv[e] = in ? rd(sp + k * HN) : 0.f;
      gv[e] = in ? rd(gp + r * HN) : 0.f;
      ds[e] = in ? rd(dp + (long long)k * a.H) : 0.f;
      dg[e] = in ? rd(dp + (long long)r * a.H) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = k0 + e, r = w.segs - 1 - k;
      if (k >= w.segs) break;
      wr(sp + k * HN, s);
      wr(gp + r * HN, g);
      s = fmaf(ex2(ds[e] * A), s, sv[e]);
      g = fmaf(ex2(dg[e] * A), g, gv[e]);
    }
  }
}

// 16 values per lane summed over the warp's channel slots: halves are exchanged over the lanes'
// highest bit first, so that a lane comes to hold 16 / SLOTS of the sums (one, twice, with 32
// slots), the k-th being value kept(k).
template <int LPC>
struct SumSlots {
  static constexpr int SLOTS = 32 / LPC, KEEP = SLOTS >= 16 ? 1 : 16 / SLOTS;
  static __device__ __forceinline__ void run(float (&r)[16], int wl) {
    int m = 8;
#pragma unroll
    for (int o = 16; o >= LPC; o >>= 1) {
      if (m == 0) {
        r[0] += __shfl_xor_sync(0xffffffffu, r[0], o);
        continue;
      }
      const bool up = wl & o;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= m) continue;
        const float keep = up ? r[i + m] : r[i], send = up ? r[i] : r[i + m];
        r[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
      m >>= 1;
    }
  }
  static __device__ __forceinline__ int kept(int wl, int k) {
    const int slot = wl / LPC;
    return SLOTS == 32 ? slot / 2 : slot * KEEP + k;
  }
  // The kept sums where at(value) says (neighbouring values are neighbours there, in fours).
  template <typename At>
  static __device__ __forceinline__ void put(const float (&r)[16], int wl, At at) {
    if constexpr (KEEP == 1) {
      *at(kept(wl, 0)) = r[0];
    } else if constexpr (KEEP == 2) {
      *reinterpret_cast<float2*>(at(kept(wl, 0))) = make_float2(r[0], r[1]);
    } else {
#pragma unroll
      for (int e = 0; e < KEEP; e += 4)
        *reinterpret_cast<float4*>(at(kept(wl, e))) = make_float4(r[e], r[e + 1], r[e + 2], r[e + 3]);
    }
  }
};

// (1 - e^-d) / d is the softplus' derivative over the softplus d.  For d < 1/2 a polynomial, the
// interpolation at the Chebyshev points of degree 4 (relative error 1e-7), which keeps the
// relative precision that 1 - e^-d loses there.
__device__ __forceinline__ float softplus_slope(float d) {
  float p = 0.006785358767956495f;
  p = fmaf(p, d, -0.041015710681676865f);
  p = fmaf(p, d, 0.16655270755290985f);
  p = fmaf(p, d, -0.4999929666519165f);
  p = fmaf(p, d, 0.9999999403953552f);
  return d < 0.5f ? p * d : 1.f - ex2(-d * kLog2e);
}

// (3) A CTA per HB channels and segment.
template <typename T, typename G, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 4) selective_tiles_kernel(s4_selective_bwd_args a, Work w, bool vec, bool vecbc,
                                                                      bool vecn, St st) {
  constexpr int LPC = G::LPC, SPT = G::SPT, CPT = G::CPT, NP = G::NP, CH = G::CH, TC = G::TC, TB = G::TB, OWN = G::OWN;
  using Sum = SumSlots<LPC>;
  extern __shared__ __align__(16) float smem[];
  float4(*steps)[G::ROW / 4] = reinterpret_cast<float4(*)[G::ROW / 4]>(smem);
  float4(*outs)[G::ROW / 4] = reinterpret_cast<float4(*)[G::ROW / 4]>(smem + TC * G::ROW);
  float(*sb)[NP] = reinterpret_cast<float(*)[NP]>(smem + G::B0);
  float(*sc)[NP] = reinterpret_cast<float(*)[NP]>(smem + G::C0);
  float4* keep = reinterpret_cast<float4*>(smem + G::S0) + threadIdx.x;
  float(*reds)[TB][G::RROW] = reinterpret_cast<float(*)[TB][G::RROW]>(smem + G::R0);  // blocks take them in turn
  const int b = blockIdx.y, seg = blockIdx.x / w.blocks, block = blockIdx.x % w.blocks;
  const int wid = threadIdx.x / 32, wl = threadIdx.x & 31;
  const Chan c = chan_of<G::HB>(block, a.H / a.G);
  const Seq q = seq_of(a.lengths, nullptr, b, a.L, 0, st);
  const Place<G> p(c.h0 + wid * CH, c.hend);
  const int lane = p.lane, n0 = p.n0, h = p.h, nh = p.nh, nn = a.N - n0, cs = wid * G::SLOTS + p.slot;
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
  const T* dt = static_cast<const T*>(a.dt.p) + b * a.dt.batch + h;
  const T* z = a.z.p ? static_cast<const T*>(a.z.p) + b * a.z.batch + h : nullptr;
  const T* dy = static_cast<const T*>(a.dy.p) + b * a.dy.batch + h;
  const T* B = static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group;
  const T* C = static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group;
  T* dxo = static_cast<T*>(a.dx.p) + b * a.dx.batch + h;
  T* dto = static_cast<T*>(a.ddt.p) + b * a.ddt.batch + h;
  T* dzo = z ? static_cast<T*>(a.dz.p) + b * a.dz.batch + h : nullptr;
  const int first = seg * w.seg_tiles, last = min(w.tiles, first + w.seg_tiles);

  // this thread's slots of the tile that comes next, the one before in time
  constexpr int V0 = 16 / (int)sizeof(T), VB = V0 < G::VECS ? V0 : G::VECS, NB = G::VECS / VB;
  Cells<T, OWN, kThreads> next{reinterpret_cast<Pack<T, 2>*>(smem + G::X0) + threadIdx.x};
  Pack<T, VB>* nextv = reinterpret_cast<Pack<T, VB>*>(smem + G::template V0<T>()) + threadIdx.x;
  float4* nexts = reinterpret_cast<float4*>(smem + G::template N0<T>()) + threadIdx.x;  // [CPT][SPT / 4][kThreads]
  const auto fetch = [&](int tile) {
    const int tb = tile * TC, live = min(TC, q.len - tb);
    if (live <= 0) return;
    const long long row = ((long long)b * w.tiles + tile) * a.H + h;
    if (WHOLE && live == TC) {
#pragma unroll
      for (int k = 0; k < OWN; ++k) next.fetch(k, a, x, dt, z, dy, tb + p.token(k));
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = (k * kThreads + threadIdx.x) * VB, t = tb + i / NP;
        if (i >= TC * NP) continue;
        fetch_whole<T, VB>(nextv + k * kThreads, B + t * a.B.row + i % NP);
        fetch_whole<T, VB>(nextv + (NB + k) * kThreads, C + t * a.C.row + i % NP);
      }
#pragma unroll
      for (int j = 0; j < CPT; ++j)
#pragma unroll
        for (int i = 0; i < SPT / 4; ++i)
          fetch_whole<float, 4>(reinterpret_cast<Pack<float, 4>*>(nexts + (j * SPT / 4 + i) * kThreads),
                                w.s_tile + (row + j) * a.N + n0 + 4 * i);
      return;
    }
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int t = p.token(k);
      next.load(k, a, x, dt, z, dy, tb + t, t < live ? p.ns : 0, vec);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = (k * kThreads + threadIdx.x) * VB, t = i / NP;
      const int n = i < TC * NP && t < live ? a.N - i % NP : 0;
      nextv[k * kThreads] = ld_pack<T, VB>(B + (long long)(tb + t) * a.B.row + i % NP, n, vecbc);
      nextv[(NB + k) * kThreads] = ld_pack<T, VB>(C + (long long)(tb + t) * a.C.row + i % NP, n, vecbc);
    }
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      float f[SPT];
      ld_f<float, SPT>(w.s_tile + (row + j) * a.N + n0, j < nh ? nn : 0, vecn, f);
#pragma unroll
      for (int i = 0; i < SPT / 4; ++i)
        nexts[(j * SPT / 4 + i) * kThreads] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
    }
  };
  fetch(last - 1);  // before the reads below, which take as long
  float2 A[CPT][SPT / 2], g[CPT][SPT / 2], dA[CPT][SPT / 2];
  float2 dD = make_float2(0.f, 0.f), db = dD;
  const float2 bias = make_float2(a.dt_bias && nh > 0 ? rd(a.dt_bias + h) : 0.f, a.dt_bias && nh > 1 ? rd(a.dt_bias + h + 1) : 0.f);
  const float2 Dv = make_float2(a.D && nh > 0 ? rd(a.D + h) : 0.f, a.D && nh > 1 ? rd(a.D + h + 1) : 0.f);
  const long long srow = ((long long)b * w.segs + seg) * a.H + h;
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int n = j < nh ? nn : 0;
    ld_states<SPT>(A[j], a.A + (long long)(h + j) * a.N + n0, n, vecn);
    if (w.segs > 1)
      ld_states<SPT>(g[j], w.g_seg + (srow + j) * a.N + n0, n, vecn);
    else
      ld_states<SPT>(g[j], a.dstate + ((long long)b * a.H + h + j) * a.N + n0, a.dstate ? n : 0, vecn);
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) {
      A[j][i] = mul2(A[j][i], make_float2(kLog2e, kLog2e));
      dA[j][i] = make_float2(0.f, 0.f);
    }
  }
  for (int tile = last - 1; tile >= first; --tile) {
    const int tb = tile * TC, live = min(TC, q.len - tb);  // <= 0: a tile of padding
    float* bc = w.part_bc + (((long long)block * a.batch + b) * a.L + tb) * 2 * NP;
    if (live <= 0) {
      const float zero[2] = {};
#pragma unroll 1
      for (int k = 0; k < OWN; ++k) {
        const int t = tb + p.token(k);
        if (t >= a.L || p.ns <= 0) continue;
        st_f<T, 2>(dxo + t * a.dx.row, p.ns, vec, zero);
        st_f<T, 2>(dto + t * a.ddt.row, p.ns, vec, zero);
        if (dzo) st_f<T, 2>(dzo + t * a.dz.row, p.ns, vec, zero);
      }
      for (int i = threadIdx.x; i < min(TC, a.L - tb) * 2 * NP; i += kThreads) wr(bc + i, 0.f);
      if (tile > first) fetch(tile - 1);
      continue;
    }
    const bool whole = WHOLE && live == TC;
    fetched();
    __syncthreads();  // the tile after this one is done with shared memory
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int t = p.token(k);
      float2 d, xv, pv, zf;
      eval_cell<T>(next.get(k, z), z != nullptr, a.softplus, bias, d, xv, pv, zf);
      if (t >= live) d = make_float2(0.f, 0.f);
      if (LPC <= 4 || lane < 4) {
        steps[t][cs] = make_float4(d.x, d.y, xv.x, xv.y);
        outs[t][cs] = make_float4(pv.x, pv.y, zf.x, zf.y);
      }
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = (k * kThreads + threadIdx.x) * VB;
      if (i >= TC * NP) continue;
      const Pack<T, VB> pb = nextv[k * kThreads], pc = nextv[(NB + k) * kThreads];
#pragma unroll
      for (int e = 0; e < VB; ++e) {
        (&sb[0][0])[i + e] = pb.get(e);
        (&sc[0][0])[i + e] = pc.get(e);
      }
    }
    // the state at the tile's start: from the segment's zero start, and what came before it
    {
      float2 s[CPT][SPT / 2];
      const long long row = ((long long)b * w.tiles + tile) * a.H + h;
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        const int n = j < nh ? nn : 0;
#pragma unroll
        for (int i = 0; i < SPT / 4; ++i) {
          const float4 v = nexts[(j * SPT / 4 + i) * kThreads];
          s[j][2 * i] = make_float2(v.x, v.y);
          s[j][2 * i + 1] = make_float2(v.z, v.w);
        }
        if (seg > 0) {
          float2 e[SPT / 2];
          ld_states<SPT>(e, w.s_seg + (srow + j) * a.N + n0, n, vecn);
          const float before = j < nh ? rd(w.d_before + row + j) : 0.f;
#pragma unroll
          for (int i = 0; i < SPT / 2; ++i)
            s[j][i] = fma2(ex2(mul2(make_float2(before, before), A[j][i])), e[i], s[j][i]);
        }
      }
      if (tile > first) fetch(tile - 1);
      __syncthreads();
      // and at the start of each block
#pragma unroll 1
      for (int k = 0;; ++k) {
#pragma unroll
        for (int i = 0; i < SPT / 2; ++i)
          keep[(k * SPT / 2 + i) * kThreads] = make_float4(s[0][i].x, s[0][i].y, s[1][i].x, s[1][i].y);
        if (k + 1 == TC / TB) break;
#pragma unroll
        for (int u = 0; u < TB; ++u) {
          const int t = k * TB + u;
          const float4 d = steps[t][cs];
          const float2 dd[CPT] = {make_float2(d.x, d.x), make_float2(d.y, d.y)};
          const float2 dx = mul2(make_float2(d.x, d.y), make_float2(d.z, d.w));
          const float2 xx[CPT] = {make_float2(dx.x, dx.x), make_float2(dx.y, dx.y)};
#pragma unroll
          for (int i = 0; i < SPT / 2; i += 2) {
            const float4 b4 = *reinterpret_cast<const float4*>(&sb[t][n0 + 2 * i]);
            const float2 bv[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int j = 0; j < CPT; ++j)
                s[j][i + e] = fma2(ex2(mul2(dd[j], A[j][i + e])), s[j][i + e], mul2(xx[j], bv[e]));
          }
        }
      }
    }
#pragma unroll 1
    for (int k = TC / TB - 1; k >= 0; --k) {
      float2 s[TB][CPT][SPT / 2];  // before each token
      float(*red)[TB][G::RROW] = reds + (k & 1) * G::WARPS;
      float vy[CPT][TB], vu[CPT][TB], vw[CPT][TB];
#pragma unroll
      for (int i = 0; i < SPT / 2; ++i) {
        const float4 v = keep[(k * SPT / 2 + i) * kThreads];
        s[0][0][i] = make_float2(v.x, v.y);
        s[0][1][i] = make_float2(v.z, v.w);
      }
      // forward: the block's states, y, and dC
      float r[16];
#pragma unroll
      for (int u = 0; u < TB; ++u) {
        const int t = k * TB + u;
        const float4 d = steps[t][cs];
        const float2 pv = *reinterpret_cast<const float2*>(&outs[t][cs]);
        const float2 dd[CPT] = {make_float2(d.x, d.x), make_float2(d.y, d.y)};
        const float2 dx = mul2(make_float2(d.x, d.y), make_float2(d.z, d.w));
        const float2 xx[CPT] = {make_float2(dx.x, dx.x), make_float2(dx.y, dx.y)};
        const float2 pp[CPT] = {make_float2(pv.x, pv.x), make_float2(pv.y, pv.y)};
        float2 y[CPT];
#pragma unroll
        for (int i = 0; i < SPT / 2; i += 2) {
          const float4 b4 = *reinterpret_cast<const float4*>(&sb[t][n0 + 2 * i]);
          const float4 c4 = *reinterpret_cast<const float4*>(&sc[t][n0 + 2 * i]);
          const float2 bv[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
          const float2 cv[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2 rc;
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
              const float2 now = fma2(ex2(mul2(dd[j], A[j][i + e])), s[u][j][i + e], mul2(xx[j], bv[e]));
              if (u + 1 < TB) s[u + 1][j][i + e] = now;
              y[j] = i + e ? fma2(cv[e], now, y[j]) : mul2(cv[e], now);
              rc = j ? fma2(pp[j], now, rc) : mul2(pp[j], now);
            }
            r[u % G::GT * SPT + 2 * (i + e)] = rc.x;
            r[u % G::GT * SPT + 2 * (i + e) + 1] = rc.y;
          }
        }
#pragma unroll
        for (int j = 0; j < CPT; ++j) vy[j][u] = y[j].x + y[j].y;
        if (u % G::GT == G::GT - 1) {  // a group's dC
          Sum::run(r, wl);
          Sum::put(r, wl, [&](int v) { return &red[wid][u - (G::GT - 1) + v / SPT][NP + n0 + v % SPT]; });
        }
      }
      // Padding adds nothing to dA, whatever state it holds back (an infinite one: 0 inf).  With 4 states
      // per thread those states are cleared (skipping each product costs 2 % on 4 x 4096 x 2048 with 16
      // states); with 8, where this spills more, the products are skipped (clearing costs 5 %).
      constexpr bool CLEAR = SPT == 4;
      if (CLEAR && !whole && (k + 1) * TB > live) {
#pragma unroll
        for (int u = 0; u < TB; ++u)
#pragma unroll
          for (int i = 0; i < SPT / 2; ++i)
            if (k * TB + u >= live) s[u][0][i] = s[u][1][i] = make_float2(0.f, 0.f);
      }
      // backward: the gradients of the states, dB, u, w, dA
#pragma unroll
      for (int u = TB - 1; u >= 0; --u) {
        const int t = k * TB + u;
        const float4 d = steps[t][cs];
        const float2 pv = *reinterpret_cast<const float2*>(&outs[t][cs]);
        const float2 dd[CPT] = {make_float2(d.x, d.x), make_float2(d.y, d.y)};
        const float2 dx = mul2(make_float2(d.x, d.y), make_float2(d.z, d.w));
        const float2 xx[CPT] = {make_float2(dx.x, dx.x), make_float2(dx.y, dx.y)};
        const float2 pp[CPT] = {make_float2(pv.x, pv.x), make_float2(pv.y, pv.y)};
        float2 uu[CPT], ww[CPT];
#pragma unroll
        for (int i = 0; i < SPT / 2; i += 2) {
          const float4 b4 = *reinterpret_cast<const float4*>(&sb[t][n0 + 2 * i]);
          const float4 c4 = *reinterpret_cast<const float4*>(&sc[t][n0 + 2 * i]);
          const float2 bv[2] = {make_float2(b4.x, b4.y), make_float2(b4.z, b4.w)};
          const float2 cv[2] = {make_float2(c4.x, c4.y), make_float2(c4.z, c4.w)};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float2 rb;
#pragma unroll
            for (int j = 0; j < CPT; ++j) {
              const float2 gv = fma2(cv[e], pp[j], g[j][i + e]);
              rb = j ? fma2(xx[j], gv, rb) : mul2(xx[j], gv);
              uu[j] = i + e ? fma2(bv[e], gv, uu[j]) : mul2(bv[e], gv);
              g[j][i + e] = mul2(gv, ex2(mul2(dd[j], A[j][i + e])));
              const float2 q1 = mul2(g[j][i + e], s[u][j][i + e]);
              ww[j] = i + e ? fma2(A[j][i + e], q1, ww[j]) : mul2(A[j][i + e], q1);
              if (CLEAR || whole || t < live) dA[j][i + e] = fma2(dd[j], q1, dA[j][i + e]);
            }
            r[u % G::GT * SPT + 2 * (i + e)] = rb.x;
            r[u % G::GT * SPT + 2 * (i + e) + 1] = rb.y;
          }
        }
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          vu[j][u] = uu[j].x + uu[j].y;
          vw[j][u] = ww[j].x + ww[j].y;
        }
        if (u % G::GT == 0) {
          Sum::run(r, wl);
          Sum::put(r, wl, [&](int v) { return &red[wid][u + v / SPT][n0 + v % SPT]; });
        }
      }
      // the block's tokens, each finished by the lane that owns it
#pragma unroll
      for (int j = 0; j < CPT; ++j) {
        sum_lanes<LPC>(vy[j], lane);
        sum_lanes<LPC>(vu[j], lane);
        sum_lanes<LPC>(vw[j], lane);
      }
#pragma unroll
      for (int i = 0; i < kOwn<LPC>; ++i) {
        const int t = k * TB + own_token<LPC>(lane, i);
        const float4 c0 = steps[t][cs], c1 = outs[t][cs];
        const float d[2] = {c0.x, c0.y}, xv[2] = {c0.z, c0.w}, pv[2] = {c1.x, c1.y}, zf[2] = {c1.z, c1.w};
        const float Dj[2] = {Dv.x, Dv.y};
        float o1[2], o2[2], o3[2], od[2];
#pragma unroll
        for (int j = 0; j < CPT; ++j) {
          o1[j] = fmaf(d[j], vu[j][i], Dj[j] * pv[j]);
          o2[j] = fmaf(xv[j], vu[j][i], kLn2 * vw[j][i]);
          if (a.softplus) o2[j] *= softplus_slope(d[j]);
          o3[j] = zf[j] * fmaf(Dj[j], xv[j], vy[j][i]);
          if (t >= live) o1[j] = o2[j] = o3[j] = 0.f;
          od[j] = pv[j] * xv[j];
        }
        dD = add2(dD, make_float2(od[0], od[1]));
        db = add2(db, make_float2(o2[0], o2[1]));
        const long long tt = tb + t;
        if (whole) {
          if (LPC <= 4 || lane < 4) {
            st_whole<T, 2>(dxo + tt * a.dx.row, o1);
            st_whole<T, 2>(dto + tt * a.ddt.row, o2);
            if (dzo) st_whole<T, 2>(dzo + tt * a.dz.row, o3);
          }
        } else if (tt < a.L && p.ns > 0) {
          st_f<T, 2>(dxo + tt * a.dx.row, p.ns, vec, o1);
          st_f<T, 2>(dto + tt * a.ddt.row, p.ns, vec, o2);
          if (dzo) st_f<T, 2>(dzo + tt * a.dz.row, p.ns, vec, o3);
        }
      }
      __syncthreads();
      for (int i = threadIdx.x; i < TB * 2 * NP; i += kThreads) {
        const int u = i / (2 * NP), n = i % (2 * NP);
        float v = 0.f;
#pragma unroll
        for (int e = 0; e < G::WARPS; ++e) v += red[e][u][n];
        const int t = k * TB + u;
        if (tb + t < a.L) wr(bc + t * 2 * NP + n, t < live ? v : 0.f);
      }
    }
  }
  // the segment's part of dA, dD, ddt_bias (lanes that own no tokens hold the sums of none)
  float* ph = w.part_h + ((long long)b * w.segs + seg) * w.pitch_h;
  if (LPC > 4 && lane >= 4) dD = db = make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 1; o < (LPC < 4 ? LPC : 4); o <<= 1) {
    dD.x += __shfl_xor_sync(0xffffffffu, dD.x, o);
    dD.y += __shfl_xor_sync(0xffffffffu, dD.y, o);
    db.x += __shfl_xor_sync(0xffffffffu, db.x, o);
    db.y += __shfl_xor_sync(0xffffffffu, db.y, o);
  }
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    if (j >= nh) continue;
    st_states<SPT>(ph + (long long)(h + j) * a.N + n0, nn, vecn, dA[j]);
    if (seg == 0 && a.dstate0) st_states<SPT>(a.dstate0 + ((long long)b * a.H + h + j) * a.N + n0, nn, vecn, g[j]);
    if (lane == 0) {
      wr(ph + (long long)a.H * a.N + h + j, j ? dD.y : dD.x);
      wr(ph + (long long)a.H * (a.N + 1) + h + j, j ? db.y : db.x);
    }
  }
}

// (4) The partial sums, in one launch: those over segments and sequences by the first CTAs, dB and dC
// over a group's channel blocks by the others.
template <typename T>
__global__ void __launch_bounds__(256) selective_sums_kernel(s4_selective_bwd_args a, Work w, int NP, int param_ctas) {
  const long long HN = (long long)a.H * a.N, cols = HN + 2ll * a.H;
  if (blockIdx.x < param_ctas) {
    column_sums(w.part_h, a.batch * w.segs, cols, w.pitch_h, [=](long long c, float v) {
      if (c < HN)
        wr(a.dA + c, v);
      else if (c < HN + a.H) {
        if (a.dD) wr(a.dD + c - HN, v);
      } else if (a.ddt_bias) {
        wr(a.ddt_bias + c - HN - a.H, v);
      }
    });
    return;
  }
  const long long i = (long long)(blockIdx.x - param_ctas) * 256 + threadIdx.x, rows = (long long)a.batch * a.L;
  const int per_row = a.G * 2 * NP, per = w.blocks / a.G;
  if (i >= rows * per_row) return;
  const long long row = i / per_row;
  const int g = (int)(i % per_row) / (2 * NP), n = (int)(i % (2 * NP)), state = n % NP;
  const float* p = w.part_bc + ((long long)g * per * rows + row) * 2 * NP + n;
  float v = 0.f;
#pragma unroll 4
  for (int k = 0; k < per; ++k) v += rd(p + (long long)k * rows * 2 * NP);
  if (state >= a.N) return;
  T* out = static_cast<T*>(n < NP ? a.dB : a.dC);
  wr(out + (row * a.G + g) * a.N + state, from_f<T>(v));
}

// The lanes that hold N states: 4 each in (3), 8 each in (1).
template <typename F>
auto with_states(int N, F f) {
  if (N <= 4) return f(Geo<1, 4>{}, EndsGeo<1, 8, Geo<1, 4>::TC>{});
  if (N <= 8) return f(Geo<2, 4>{}, EndsGeo<1, 8, Geo<2, 4>::TC>{});
  if (N <= 16) return f(Geo<4, 4>{}, EndsGeo<2, 8, Geo<4, 4>::TC>{});
  if (N <= 32) return f(Geo<8, 4>{}, EndsGeo<4, 8, Geo<8, 4>::TC>{});
  if (N <= 64) return f(Geo<16, 4>{}, EndsGeo<8, 8, Geo<16, 4>::TC>{});
  if (N <= 128) return f(Geo<32, 4>{}, EndsGeo<16, 8, Geo<32, 4>::TC>{});
  return f(Geo<32, 8>{}, EndsGeo<32, 8, Geo<32, 8>::TC>{});
}

// CTAs per SM that the segments are meant to give: six rounds of (3).  4 sequences of 4096 tokens, 2048
// channels and 16 states took 920 us with four rounds, 900 with six; 2 of 333 tokens, 256
// channels and 64 states 127 us with segments of four tiles or more, 65 with one.
constexpr int kCtas = 24;

// Sizes and the workspace's layout (pointers relative to a null base when ws is null).
template <typename G>
Work layout(int batch, int L, int H, int N, int Gr, char* ws, size_t* total) {
  Work w;
  w.tiles = (L + G::TC - 1) / G::TC;
  w.blocks = chan_blocks<G::HB>(H, Gr);
  const long long ctas = (long long)batch * w.blocks, want = (long long)s4impl::num_sms() * kCtas;
  long long segs = (want + ctas - 1) / ctas;
  if (segs > w.tiles) segs = w.tiles;
  w.seg_tiles = (int)((w.tiles + segs - 1) / segs);
  w.segs = (w.tiles + w.seg_tiles - 1) / w.seg_tiles;
  const size_t HN = (size_t)H * N, bt = (size_t)batch * w.tiles, bs = (size_t)batch * w.segs;
  size_t at = s4impl::kStatusBytes;
  auto take = [&](size_t n) {
    float* p = reinterpret_cast<float*>(ws + at);
    at += s4impl::align256(4 * n) + s4impl::kGap;
    return p;
  };
  w.s_tile = take(bt * HN);
  w.d_before = take(bt * H);
  w.s_seg = take(bs * HN);
  w.g_seg = take(bs * HN);
  w.d_seg = take(bs * H);
  w.pitch_h = ((long long)H * (N + 2) + 3) / 4 * 4;
  w.part_h = take(bs * w.pitch_h);
  w.part_bc = take((size_t)w.blocks * batch * L * 2 * G::NP);
  // CTAs of one launch
  if (total) *total = (long long)chan_blocks<2>(H, Gr) * w.segs > INT_MAX ? 0 : at;
  return w;
}

#ifdef S4_BOUNDS_CHECK
cudaError_t extents(const s4_selective_bwd_args& a, const Work& w, int NP, int e, cudaStream_t s) {
  s4impl::Extents x{};
  const long long b = a.batch, H = a.H, N = a.N;
  for (const s4_rows* r : {&a.x, &a.dt, &a.z, &a.dy}) x.in_rows(*r, e, a.batch, a.L, H);
  x.add(a.B.p, e, true, false, N, b, a.B.batch, a.L, a.B.row, a.G, a.B_group);
  x.add(a.C.p, e, true, false, N, b, a.C.batch, a.L, a.C.row, a.G, a.C_group);
  for (const s4_rows_out* r : {&a.dx, &a.ddt, &a.dz}) x.out_rows(*r, e, a.batch, a.L, H);
  for (const void* p : {a.dB, a.dC}) x.out(p, e, N, b * a.L * a.G);
  x.in(a.A, 4, N, H);
  for (const float* p : {a.D, a.dt_bias}) x.in(p, 4, H);
  x.in(a.lengths, 4, b);
  for (const float* p : {a.state0, a.dstate}) x.in(p, 4, N, b * H);
  x.out(a.dstate0, 4, N, b * H);
  x.out(a.dA, 4, N, H);
  for (const float* p : {a.dD, a.ddt_bias}) x.out(p, 4, H);
  x.scratch(w.s_tile, 4, N, b * w.tiles * H);
  x.scratch(w.d_before, 4, H, b * w.tiles);
  for (const float* p : {w.s_seg, w.g_seg}) x.scratch(p, 4, N, b * w.segs * H);
  x.scratch(w.d_seg, 4, H, b * w.segs);
  x.add(w.part_h, 4, true, true, H * (N + 2), b * w.segs, w.pitch_h);
  x.scratch(w.part_bc, 4, 2 * NP, (long long)w.blocks * b * a.L);
  return set_extents(x, s);
}
#endif

template <typename T>
cudaError_t bwd_t(const s4_selective_bwd_args& a, St st, cudaStream_t s) {
  const int e = sizeof(T);
  with_states(a.N, [&](auto geo, auto egeo) {
    using G = decltype(geo);
    using E = decltype(egeo);
    const auto ok = [&](const auto& r) { return vec_ok(r.p, e, 2 * e, r.batch, r.row); };
    const bool vec = ok(a.x) && ok(a.dt) && ok(a.z) && ok(a.dy) && ok(a.dx) && ok(a.ddt) && ok(a.dz) &&
                     (a.G == 1 || (a.H / a.G) % 2 == 0);
    constexpr int pb = e * (16 / e < E::VECS ? 16 / e : E::VECS);
    const bool vecbc = vec_ok(a.B.p, e, pb, a.B.batch, a.B.row) && vec_ok(a.C.p, e, pb, a.C.batch, a.C.row) &&
                       a.B_group * e % pb == 0 && a.C_group * e % pb == 0;
    const bool vecn = a.N % 4 == 0 && vec_ok(a.A, 4, 16) && vec_ok(a.state0, 4, 16) && vec_ok(a.dstate, 4, 16) &&
                      vec_ok(a.dstate0, 4, 16);
    const Work w = layout<G>(a.batch, a.L, a.H, a.N, a.G, static_cast<char*>(a.ws), nullptr);
#ifdef S4_BOUNDS_CHECK
    if (extents(a, w, G::NP, e, s) != cudaSuccess) return;
#endif
    const auto run = [&](auto whole) {
      constexpr bool W = decltype(whole)::value;
      constexpr auto ends = selective_ends_kernel<T, E, W>;
      constexpr auto tiles = selective_tiles_kernel<T, G, W>;
      allow_shared<ends>(E::kBytes);
      allow_shared<tiles>(G::template kBytes<T>());
      {
        s4impl::TimedLaunch tl("selective_bwd", s);
        const long long tasks = (long long)chan_blocks<E::CH>(a.H, a.G) * w.segs;
        ends<<<dim3((unsigned)((tasks + G::WARPS - 1) / G::WARPS), a.batch), kThreads, E::kBytes, s>>>(a, w, vec, vecbc,
                                                                                                       vecn, st);
      }
      if (w.segs > 1) {
        s4impl::TimedLaunch tl("selective_bwd", s);
        const long long HN = (long long)a.H * a.N;
        selective_joins_kernel<<<dim3((unsigned)((HN + 127) / 128), a.batch), 128, 0, s>>>(a, w);
      }
      s4impl::TimedLaunch tl("selective_bwd", s);
      tiles<<<dim3((unsigned)(w.blocks * w.segs), a.batch), kThreads, G::template kBytes<T>(), s>>>(a, w, vec, vecbc, vecn, st);
    };
    // Whole tiles spare a condition per access and overlap the next tile's copies: 4 sequences of 2048 tokens and 1024
    // channels (bfloat16) take 266, 302 and 548 us instead of 485, 486 and 793 with 8, 16 and 32 states.  They are
    // compiled for these numbers only; with 64, 128 and 256 states the same takes 1.71, 4.85 and 15.9 ms and
    // would take 1.26, 3.61 and 11.1.
    bool whole = false;
    if constexpr (G::LPC <= 8 && (int)G::NP == (int)E::NP) {
      whole = vec && vecbc && a.N == G::NP && (a.H / a.G) % G::HB == 0;
      if (whole) run(std::true_type{});
    }
    if (!whole) run(std::false_type{});
    s4impl::TimedLaunch tl("selective_bwd", s);
    const int param_ctas = (int)(((long long)a.H * (a.N + 2) + 31) / 32);
    const long long n = (long long)a.batch * a.L * a.G * 2 * G::NP;
    selective_sums_kernel<T><<<(unsigned)(param_ctas + (n + 255) / 256), 256, 0, s>>>(a, w, G::NP, param_ctas);
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
  with_states(N, [&](auto geo, auto) { layout<decltype(geo)>(batch, L, H, N, G, nullptr, &total); });
  return total;
}

cudaError_t launch_selective_bwd(const s4_selective_bwd_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float>(a, st, s);
  if (a.dtype == S4_BF16) return bwd_t<__nv_bfloat16>(a, st, s);
  return bwd_t<__half>(a, st, s);
}

}  // namespace s4impl
