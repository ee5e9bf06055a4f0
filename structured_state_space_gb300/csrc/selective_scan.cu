// The selective state-space scan, forward: prompts and single tokens.
//
//   d = softplus(dt + dt_bias),  s_n = 2^(d A_n log2 e) s_n + d x B_n,  y = (sum_n C_n s_n + D x) silu(z)
//
// Per (token, channel, state): one exponential (the SM's special function units give 32 of them
// a clock) and four multiplications or additions (128 a clock), so that both pipes need 4
// clocks of an SM quarter for 32 of them; the activations are 8 bytes per (token, channel) in
// 16 bits.  At N = 16 the exponentials bound it, not memory.
//
// The recurrence is sequential in time, parallel over sequences, channels and states.  A warp
// takes CH channels and walks a stretch of tokens.  Where there are too few channels to fill the GPU, the
// tokens are split into chunks: a first kernel gives each chunk's state from a zero start
// and its total step (which fixes its decay), a second joins them, the third runs the chunks
// from their true starts.  That costs the exponentials twice.
//
// Measured (bfloat16, 16 states): 560 us for one sequence of 65536 tokens and 1024 channels, 215 of them
// for the chunks' ends, against 115 us of exponentials per pass and 337 us for both inner loops in
// registers alone; 57 % of the issue slots are used at 16 warps per SM.
#include "selective.cuh"

namespace {
using namespace s4sel;

// Four CTAs of four warps per SM: 128 registers a thread.  At 20 warps per SM the registers
// left do not hold enough exponentials in flight (650 us instead of 564 on one sequence of
// 65536 tokens, 1024 channels, 16 states, bfloat16), at 14 there are too few warps (647 us).
constexpr int kScanThreads = 128, kScanCtas = 4, kStepThreads = 128;

template <int LPC_, int SPT_>
struct Geo {
  static constexpr int LPC = LPC_, SPT = SPT_, NP = LPC * SPT, CPT = 2;
  static constexpr int CH = 32 / LPC * CPT;              // channels of a warp
  static constexpr int TT = NP <= 64 ? 8 : 4;            // tokens of a tile
  static constexpr int OWN = TT / 4 * kOwn<LPC>;         // tokens of a tile that a lane stages and finishes
  static constexpr int VECS = TT * NP / 32;              // elements of B, of C that a lane stages
  // Shared memory of a warp in floats: steps and step x of channel pairs [TT][DROW] | B | C [TT][NP]
  // | the next tile's x, dt, z [3][OWN][32] packs of 2 | its B, C
  static constexpr int DROW = 128 / LPC + row_pad(LPC, 128 / LPC);
  static constexpr int B0 = TT * DROW, C0 = B0 + TT * NP, X0 = C0 + TT * NP;
  static constexpr int V0 = X0 + 3 * OWN * 32 * 2, END = V0 + 2 * TT * NP;
  static constexpr int kBytes = 4 * END * (kScanThreads / 32);
};

struct Chunks {
  int len, count;   // tokens per chunk (a multiple of the tile), number of chunks
  float *start;     // [batch][count][H][N]: end states from zero, then start states
  float *total;     // [batch][count][H]: sums of the step sizes
};

// MODE 0: states from a zero start and total steps of chunks 0 .. count - 2; MODE 1: outputs.
//
// Warps work alone: a lane stages the step sizes of its 2 channels for the tokens it owns, the
// LPC lanes of the channels read them back, and after the sums over these lanes the same lane
// holds y of the same tokens, beside their x and z.  So only (step, step x) and the vectors B
// and C pass through shared memory, and no barrier is wider than a warp.  Shared memory delivers
// 32 words a clock to the registers of an SM, broadcast or not, and an exponential takes 1/32
// clock: 8 states by 2 channels per thread read 20 words for 16 exponentials, at 16 warps per SM.
//
// WHOLE: every access is aligned and every warp's channels and states exist, so that tiles of real
// tokens are read and written without a condition.
template <typename T, typename G, int MODE, bool WHOLE>
__global__ void __launch_bounds__(kScanThreads, kScanCtas)
    selective_scan_kernel(s4_selective_args a, Chunks ck, bool vec, bool vecbc, St st) {
  constexpr int LPC = G::LPC, SPT = G::SPT, NP = G::NP, CH = G::CH, TT = G::TT, CPT = G::CPT, OWN = G::OWN;
  constexpr int V0 = 16 / (int)sizeof(T), VB = V0 < G::VECS ? V0 : G::VECS, NB = G::VECS / VB;
  extern __shared__ __align__(16) float smem[];
  float* mine = smem + threadIdx.x / 32 * G::END;
  float4(*sd)[G::DROW / 4] = reinterpret_cast<float4(*)[G::DROW / 4]>(mine);
  float(*sb)[NP] = reinterpret_cast<float(*)[NP]>(mine + G::B0);
  float(*sc)[NP] = reinterpret_cast<float(*)[NP]>(mine + G::C0);
  record_gen(st);
  const int b = blockIdx.z, wl = threadIdx.x & 31;
  const int blocks = chan_blocks<CH>(a.H, a.G), count = MODE ? ck.count : ck.count - 1;
  const long long task = (long long)blockIdx.x * (kScanThreads / 32) + threadIdx.x / 32;
  const Seq q = seq_of(a.lengths, a.index, b, a.L, a.slots, st);
  if (task >= (long long)blocks * count) return;
  const int chunk = (int)(task / blocks);
  const Chan c = chan_of<CH>((int)(task % blocks), a.H / a.G);
  const int t0 = chunk * ck.len, t1 = min(a.L, t0 + ck.len), live = min(t1, q.len);
  if (MODE == 0 && t0 >= q.len) return;
  const int lane = wl % LPC, slot = wl / LPC, n0 = lane * SPT, h = c.h0 + slot * CPT, nh = c.hend - h;
  const int ns = LPC > 4 && lane >= 4 ? 0 : nh;  // channels this lane stages and finishes
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
  const T* dt = static_cast<const T*>(a.dt.p) + b * a.dt.batch + h;
  const T* z = MODE && a.z.p ? static_cast<const T*>(a.z.p) + b * a.z.batch + h : nullptr;
  const T* B = static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group;
  const T* C = static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group;
  T* y = MODE ? static_cast<T*>(a.y.p) + b * a.y.batch + h : nullptr;

  // the k-th token of a tile that this lane owns
  const auto token = [&](int k) { return k / kOwn<LPC> * 4 + own_token<LPC>(lane, k % kOwn<LPC>); };
  // this lane's slots of the next tile
  Pack<T, CPT>* next = reinterpret_cast<Pack<T, CPT>*>(mine + G::X0) + wl;
  Pack<T, VB>* nextv = reinterpret_cast<Pack<T, VB>*>(mine + G::V0) + wl;
  const auto fetch = [&](int tb) {
    if (WHOLE && tb + TT <= live) {
#pragma unroll
      for (int k = 0; k < OWN; ++k) {
        const int t = tb + token(k);
        fetch_whole<T, CPT>(next + k * 32, x + t * a.x.row);
        fetch_whole<T, CPT>(next + (OWN + k) * 32, dt + t * a.dt.row);
        if (z) fetch_whole<T, CPT>(next + (2 * OWN + k) * 32, z + t * a.z.row);
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = (k * 32 + wl) * VB, t = tb + i / NP;
        fetch_whole<T, VB>(nextv + k * 32, B + t * a.B.row + i % NP);
        if (MODE == 1) fetch_whole<T, VB>(nextv + (NB + k) * 32, C + t * a.C.row + i % NP);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      const int t = tb + token(k), n = t < live ? ns : 0;
      next[k * 32] = ld_pack<T, CPT>(x + t * a.x.row, n, vec);
      next[(OWN + k) * 32] = ld_pack<T, CPT>(dt + t * a.dt.row, n, vec);
      if (z) next[(2 * OWN + k) * 32] = ld_pack<T, CPT>(z + t * a.z.row, n, vec);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = (k * 32 + wl) * VB, t = tb + i / NP;
      const int n = t < live ? a.N - i % NP : 0;
      nextv[k * 32] = ld_pack<T, VB>(B + t * a.B.row + i % NP, n, vecbc);
      if (MODE == 1) nextv[(NB + k) * 32] = ld_pack<T, VB>(C + t * a.C.row + i % NP, n, vecbc);
    }
  };
  if (t0 < live) fetch(t0);  // before the reads below, which take as long
  float2 A[CPT][SPT / 2], s[CPT][SPT / 2];  // pairs of neighbouring states
  float bias[CPT], skip[CPT];
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < CPT; ++j) {
    const int hs = h + j;
    const bool on = j < nh;
    bias[j] = a.dt_bias && on ? rd(a.dt_bias + hs) : 0.f;
    skip[j] = MODE && a.D && on ? rd(a.D + hs) : 0.f;
#pragma unroll
    for (int i = 0; i < SPT; ++i) {
      const int n = n0 + i;
      const bool in = on && n < a.N;
      float v = 0.f;
      if (MODE == 1 && in && (t0 < q.len || chunk == 0)) {
        if (ck.count > 1)
          v = rd(ck.start + (((long long)b * ck.count + chunk) * a.H + hs) * a.N + n);
        else if (a.state && q.slot >= 0)
          v = rd(a.state + (q.slot * a.H + hs) * a.N + n);
      }
      const float Av = in ? rd(a.A + (long long)hs * a.N + n) * kLog2e : 0.f;
      (i % 2 ? A[j][i / 2].y : A[j][i / 2].x) = Av;
      (i % 2 ? s[j][i / 2].y : s[j][i / 2].x) = v;
    }
  }

  for (int tb = t0; tb < live; tb += TT) {
    const bool whole = tb + TT <= live;
    Pack<T, CPT> px[OWN], pz[OWN];
    fetched();
    __syncwarp();  // the tile before has been read
#pragma unroll
    for (int k = 0; k < OWN; ++k) {
      px[k] = next[k * 32];
      if (z) pz[k] = next[(2 * OWN + k) * 32];
      const Pack<T, CPT> pd = next[(OWN + k) * 32];
      float2 d = make_float2(pd.get(0) + bias[0], pd.get(1) + bias[1]);
      if (a.softplus) d = softplus2(d);
      if (!whole && tb + token(k) >= live) d = make_float2(0.f, 0.f);  // padding keeps the state
      const float2 dx = mul2(d, make_float2(px[k].get(0), px[k].get(1)));
      if (MODE == 0) sum = add2(sum, d);
      if (LPC <= 4 || lane < 4) sd[token(k)][slot] = make_float4(d.x, d.y, dx.x, dx.y);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = (k * 32 + wl) * VB;
      const Pack<T, VB> pb = nextv[k * 32];
#pragma unroll
      for (int e = 0; e < VB; ++e) (&sb[0][0])[i + e] = pb.get(e);
      if (MODE == 1) {
        const Pack<T, VB> pc = nextv[(NB + k) * 32];
#pragma unroll
        for (int e = 0; e < VB; ++e) (&sc[0][0])[i + e] = pc.get(e);
      }
    }
    __syncwarp();
    if (tb + TT < live) fetch(tb + TT);
#pragma unroll
    for (int u = 0; u < TT; u += 4) {
      float v[CPT][4];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float4 d = sd[u + w][slot];
        const float2 dd[CPT] = {make_float2(d.x, d.x), make_float2(d.y, d.y)};
        const float2 xx[CPT] = {make_float2(d.z, d.z), make_float2(d.w, d.w)};
        float2 acc[CPT];
#pragma unroll
        for (int i = 0; i < SPT / 2; i += 2) {
          const float4 b4 = *reinterpret_cast<const float4*>(&sb[u + w][n0 + 2 * i]);
          const float2 b0 = make_float2(b4.x, b4.y), b1 = make_float2(b4.z, b4.w);
          float2 c0, c1;
          if (MODE == 1) {
            const float4 c4 = *reinterpret_cast<const float4*>(&sc[u + w][n0 + 2 * i]);
            c0 = make_float2(c4.x, c4.y);
            c1 = make_float2(c4.z, c4.w);
          }
#pragma unroll
          for (int j = 0; j < CPT; ++j) {
            s[j][i] = fma2(ex2(mul2(dd[j], A[j][i])), s[j][i], mul2(xx[j], b0));
            s[j][i + 1] = fma2(ex2(mul2(dd[j], A[j][i + 1])), s[j][i + 1], mul2(xx[j], b1));
            if (MODE == 1) {
              acc[j] = i ? fma2(c0, s[j][i], acc[j]) : mul2(c0, s[j][i]);
              acc[j] = fma2(c1, s[j][i + 1], acc[j]);
            }
          }
        }
        if (MODE == 1) {
#pragma unroll
          for (int j = 0; j < CPT; ++j) v[j][w] = acc[j].x + acc[j].y;
        }
      }
      if (MODE == 1) {
        // y of four tokens, finished by the lanes that own them: skip term, gate, one rounding
#pragma unroll
        for (int j = 0; j < CPT; ++j) sum_lanes<LPC>(v[j], lane);
#pragma unroll
        for (int i = 0; i < kOwn<LPC>; ++i) {
          const int k = u / 4 * kOwn<LPC> + i, t = tb + token(k);
          float out[CPT];
#pragma unroll
          for (int j = 0; j < CPT; ++j) {
            out[j] = fmaf(skip[j], px[k].get(j), v[j][i]);
            if (z) out[j] *= silu(pz[k].get(j));
          }
          if (WHOLE && whole) {
            if (LPC <= 4 || lane < 4) st_whole<T, CPT>(y + t * a.y.row, out);
          } else if (t < live && ns > 0) {
            st_f<T, CPT>(y + t * a.y.row, ns, vec, out);
          }
        }
      }
    }
  }
  if (MODE == 1) {  // padding
    const float zero[CPT] = {};
    for (int t = max(t0, live) + lane; t < t1; t += LPC)
      if (nh > 0) st_f<T, CPT>(y + t * a.y.row, nh, vec, zero);
  }
  // Where the state goes: the chunk's end state, or, after the last real token, the caller's slot.
  float* out = nullptr;
  if (MODE == 0)
    out = ck.start + ((long long)b * ck.count + chunk) * a.H * a.N;
  else if (a.state_out && q.slot >= 0 && ((t0 < q.len && q.len <= t1) || (q.len == 0 && chunk == 0)))
    out = a.state_out + q.slot * a.H * a.N;
  if (MODE == 0) {  // the tokens are spread over up to four lanes
#pragma unroll
    for (int o = 1; o < (LPC < 4 ? LPC : 4); o <<= 1) {
      sum.x += __shfl_xor_sync(0xffffffffu, sum.x, o);
      sum.y += __shfl_xor_sync(0xffffffffu, sum.y, o);
    }
  }
  if (out) {
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const int hs = h + j;
      if (j >= nh) continue;
#pragma unroll
      for (int i = 0; i < SPT; ++i)
        if (n0 + i < a.N) wr(out + (long long)hs * a.N + n0 + i, i % 2 ? s[j][i / 2].y : s[j][i / 2].x);
      if (MODE == 0 && lane == 0) wr(ck.total + ((long long)b * ck.count + chunk) * a.H + hs, j ? sum.y : sum.x);
    }
  }
}

// Joins the chunks: start_{c+1} = 2^(A total_c) start_c + end_c, in place of the end states.  A
// thread per state; 8 chunks' loads are under way at a time.
__global__ void __launch_bounds__(128) selective_join_kernel(s4_selective_args a, Chunks ck, St st) {
  const int b = blockIdx.y;
  const Seq q = seq_of(a.lengths, a.index, b, a.L, a.slots, st);
  const long long i = (long long)blockIdx.x * 128 + threadIdx.x, HN = (long long)a.H * a.N;
  if (i >= HN) return;
  const float A = rd(a.A + i) * kLog2e;
  float* p = ck.start + (long long)b * ck.count * HN + i;
  const float* tot = ck.total + (long long)b * ck.count * a.H + i / a.N;
  const int used = q.len ? (q.len + ck.len - 1) / ck.len : 1;  // chunks with real tokens
  float s = a.state && q.slot >= 0 ? rd(a.state + q.slot * HN + i) : 0.f;
  for (int c0 = 0; c0 < used; c0 += 8) {
    float end[8], d[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool more = c0 + k + 1 < used;
      end[k] = more ? rd(p + (c0 + k) * HN) : 0.f;
      d[k] = more ? rd(tot + (long long)(c0 + k) * a.H) : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (c0 + k < used) wr(p + (c0 + k) * HN, s);
      s = fmaf(ex2(d[k] * A), s, end[k]);
    }
  }
}

// One token per sequence: the state is read, advanced and written once (8 bytes per channel and
// state, which bound it).  A thread takes 8 states of a channel and has all its reads under way
// before the first is used.  WHOLE: aligned, and every thread's channel and states exist (a
// call is then half of the instructions).  Two and four channels per thread were no faster (24.0
// us instead of 23.3 on 256 sequences of 2048 channels and 16 states, 31.5 with four, each
// launched on states out of cache; one after the other, states in cache, they take 12.7 us).
template <typename T, int LPC, int SPT, bool WHOLE>
__global__ void __launch_bounds__(kStepThreads) selective_step_kernel(s4_selective_args a, bool vec, bool vecbc, St st) {
  constexpr int HB = kStepThreads / LPC;
  record_gen(st);
  const int b = blockIdx.y;
  const Chan c = chan_of<HB>(blockIdx.x, a.H / a.G);
  const Seq q = seq_of(a.lengths, a.index, b, 1, a.slots, st);
  const int lane = threadIdx.x % LPC, h = c.h0 + threadIdx.x / LPC, n0 = lane * SPT, n = WHOLE ? SPT : a.N - n0;
  const bool in = WHOLE || h < c.hend, on = q.len > 0;  // `on`: the token advances the state
  const bool put = in && (WHOLE || n > 0) && a.state_out && q.slot >= 0;
  T* y = static_cast<T*>(a.y.p) + b * a.y.batch;
  if (WHOLE && !on && !put) {  // a row that is not in use
    if (lane == 0) wr(y + h, from_f<T>(0.f));
    return;
  }
  const long long at = (q.slot * a.H + h) * a.N + n0;
  Pack<float, SPT> ps, pA;
  Pack<T, SPT> pb, pc;
  ps.zero();
  if (in && q.slot >= 0 && a.state)
    ps = ld_pack<float, SPT>(a.state + at, n, WHOLE || vec);
  pA = ld_pack<float, SPT>(a.A + (long long)h * a.N + n0, in ? n : 0, WHOLE || vec);
  float xv = 0.f, d = 0.f, zv = 0.f;
  if (in && on) {
    xv = to_f(rd(static_cast<const T*>(a.x.p) + b * a.x.batch + h));
    d = to_f(rd(static_cast<const T*>(a.dt.p) + b * a.dt.batch + h));
    if (a.z.p) zv = to_f(rd(static_cast<const T*>(a.z.p) + b * a.z.batch + h));
  }
  pb = ld_pack<T, SPT>(static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group + n0, on ? n : 0, WHOLE || vecbc);
  pc = ld_pack<T, SPT>(static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group + n0, on ? n : 0, WHOLE || vecbc);
  if (a.dt_bias && in) d += rd(a.dt_bias + h);
  const float skip = a.D && in ? rd(a.D + h) : 0.f;

  float2 s[SPT / 2], acc = make_float2(0.f, 0.f);
  to_pairs<float, SPT>(ps, s);
  if (on) {
    float2 A[SPT / 2], Bv[SPT / 2], Cv[SPT / 2];
    to_pairs<float, SPT>(pA, A);
    to_pairs<T, SPT>(pb, Bv);
    to_pairs<T, SPT>(pc, Cv);
    if (a.softplus) d = softplus(d);
    const float2 dl = make_float2(d * kLog2e, d * kLog2e), dx = make_float2(d * xv, d * xv);
#pragma unroll
    for (int i = 0; i < SPT / 2; ++i) {
      s[i] = fma2(ex2(mul2(dl, A[i])), s[i], mul2(dx, Bv[i]));
      acc = fma2(Cv[i], s[i], acc);
    }
  }
  if (put) st_pairs<float, SPT>(a.state_out + at, n, WHOLE || vec, s);
  float v = acc.x + acc.y;
#pragma unroll
  for (int o = LPC / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (lane == 0 && in) {
    v = fmaf(skip, xv, v);
    if (a.z.p) v *= silu(zv);
    wr(y + h, from_f<T>(on ? v : 0.f));
  }
}

// Chunks: kWarps warps per SM (two rounds of what runs at once: with one, ragged sequences leave
// SMs idle, 105 us instead of 96 on four sequences of up to 1500 tokens, 2048 channels; with
// more, the joins grow), none shorter than kMinChunk tokens, and only where one chunk
// would leave more than half of a round missing (chunks take the exponentials twice).
constexpr int kWarps = 32, kMinChunk = 64, kTile = 8;
Chunks plan(int batch, int L, int H, int N, int G, int CH) {
  const long long warps = (long long)batch * G * ((H / G + CH - 1) / CH);
  const long long want = (long long)s4impl::num_sms() * kWarps;
  Chunks ck{L, 1, nullptr, nullptr};
  if (4 * warps > want || L < 2 * kMinChunk) return ck;
  long long n = want / warps;
  if (n > L / kMinChunk) n = L / kMinChunk;
  ck.len = (int)(((L + n - 1) / n + kTile - 1) / kTile * kTile);
  ck.count = (L + ck.len - 1) / ck.len;
  return ck;
}

// The lanes that hold N states, 8 each.
template <typename F>
auto with_states(int N, F f) {
  if (N <= 8) return f(Geo<1, 8>{});
  if (N <= 16) return f(Geo<2, 8>{});
  if (N <= 32) return f(Geo<4, 8>{});
  if (N <= 64) return f(Geo<8, 8>{});
  if (N <= 128) return f(Geo<16, 8>{});
  return f(Geo<32, 8>{});
}
#ifdef S4_BOUNDS_CHECK
cudaError_t extents(const s4_selective_args& a, const Chunks& ck, int e, cudaStream_t s) {
  s4impl::Extents x{};
  for (const s4_rows* r : {&a.x, &a.dt, &a.z}) x.in_rows(*r, e, a.batch, a.L, a.H);
  x.add(a.B.p, e, true, false, a.N, a.batch, a.B.batch, a.L, a.B.row, a.G, a.B_group);
  x.add(a.C.p, e, true, false, a.N, a.batch, a.C.batch, a.L, a.C.row, a.G, a.C_group);
  x.out_rows(a.y, e, a.batch, a.L, a.H);
  x.in(a.A, 4, a.N, a.H);
  for (const float* p : {a.D, a.dt_bias}) x.in(p, 4, a.H);
  for (const int* p : {a.lengths, a.index}) x.in(p, 4, a.batch);
  x.in(a.state, 4, a.N, (long long)a.slots * a.H);
  x.out(a.state_out, 4, a.N, (long long)a.slots * a.H);
  if (ck.count > 1) {
    x.scratch(ck.start, 4, a.N, (long long)a.batch * ck.count * a.H);
    x.scratch(ck.total, 4, a.H, (long long)a.batch * ck.count);
  }
  return set_extents(x, s);
}
#endif
template <typename T>
cudaError_t step_t(const s4_selective_args& a, St st, cudaStream_t s) {
  const int e = sizeof(T);
#ifdef S4_BOUNDS_CHECK
  if (const cudaError_t err = extents(a, Chunks{1, 1, nullptr, nullptr}, e, s); err != cudaSuccess) return err;
#endif
  s4impl::TimedLaunch tl("selective_step", s);
  with_states(a.N, [&](auto geo) {
    using G = decltype(geo);
    constexpr int LPC = G::LPC, SPT = G::SPT, HB = kStepThreads / LPC, pb = e * SPT < 16 ? e * SPT : 16;
    const bool vec = a.N % 4 == 0 && vec_ok(a.state, 4, 16) && vec_ok(a.state_out, 4, 16) && vec_ok(a.A, 4, 16);
    const bool vecbc = vec_ok(a.B.p, e, pb, a.B.batch) && vec_ok(a.C.p, e, pb, a.C.batch) && a.B_group * e % pb == 0 &&
                       a.C_group * e % pb == 0;
    const dim3 grid(chan_blocks<HB>(a.H, a.G), a.batch);
    if (vec && vecbc && a.N == G::NP && (a.H / a.G) % HB == 0)
      selective_step_kernel<T, LPC, SPT, true><<<grid, kStepThreads, 0, s>>>(a, vec, vecbc, st);
    else
      selective_step_kernel<T, LPC, SPT, false><<<grid, kStepThreads, 0, s>>>(a, vec, vecbc, st);
  });
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_t(const s4_selective_args& a, St st, cudaStream_t s) {
  if (a.L == 1) return step_t<T>(a, st, s);
  const int e = sizeof(T);
  with_states(a.N, [&](auto geo) {
    using G = decltype(geo);
    constexpr int px = e * G::CPT, pb = e * (16 / e < G::VECS ? 16 / e : G::VECS), per = kScanThreads / 32;
    const auto ok = [&](const auto& r) { return vec_ok(r.p, e, px, r.batch, r.row); };
    const bool vec = ok(a.x) && ok(a.dt) && ok(a.z) && ok(a.y) && (a.G == 1 || (a.H / a.G) % G::CPT == 0);
    const bool vecbc = vec_ok(a.B.p, e, pb, a.B.batch, a.B.row) && vec_ok(a.C.p, e, pb, a.C.batch, a.C.row) &&
                       a.B_group * e % pb == 0 && a.C_group * e % pb == 0;
    Chunks ck = plan(a.batch, a.L, a.H, a.N, a.G, G::CH);
    ck.start = reinterpret_cast<float*>(static_cast<char*>(a.ws) + s4impl::kStatusBytes);
    ck.total = ck.start + (long long)a.batch * ck.count * a.H * a.N + s4impl::kGap / 4;
#ifdef S4_BOUNDS_CHECK
    if (extents(a, ck, e, s) != cudaSuccess) return;
#endif
    const long long blocks = chan_blocks<G::CH>(a.H, a.G);
    const auto run = [&](auto whole) {
      constexpr bool W = decltype(whole)::value;
      constexpr auto ends = selective_scan_kernel<T, G, 0, W>, out = selective_scan_kernel<T, G, 1, W>;
      allow_shared<ends>(G::kBytes);
      allow_shared<out>(G::kBytes);
      if (ck.count > 1) {
        {
          s4impl::TimedLaunch tl("selective_scan", s);
          const dim3 grid((unsigned)((blocks * (ck.count - 1) + per - 1) / per), 1, a.batch);
          ends<<<grid, kScanThreads, G::kBytes, s>>>(a, ck, vec, vecbc, st);
        }
        s4impl::TimedLaunch tl("selective_scan", s);
        const long long HN = (long long)a.H * a.N;
        selective_join_kernel<<<dim3((unsigned)((HN + 127) / 128), a.batch), 128, 0, s>>>(a, ck, st);
      }
      s4impl::TimedLaunch tl("selective_scan", s);
      const dim3 grid((unsigned)((blocks * ck.count + per - 1) / per), 1, a.batch);
      out<<<grid, kScanThreads, G::kBytes, s>>>(a, ck, vec, vecbc, st);
    };
    // Whole tiles spare a condition per access and overlap the next tile's copies: one sequence of 65536 tokens,
    // 1024 channels and 16 states (bfloat16) takes 592 us instead of 1479, 4 of 2048 tokens 111, 127 and 171 us
    // instead of 238, 254 and 278 with 8, 16 and 32 states.  They are compiled for up to 32 states only; with 64, 128
    // and 256 the same 4 x 2048 x 1024 takes 594, 1473 and 4598 us and would take 369, 870 and 2423.
    bool whole = false;
    if constexpr (G::LPC <= 4) {
      whole = vec && vecbc && a.N == G::NP && (a.H / a.G) % G::CH == 0;
      if (whole) run(std::true_type{});
    }
    if (!whole) run(std::false_type{});
  });
  return cudaGetLastError();
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_selective)
#endif

size_t selective_scratch(int batch, int L, int H, int N, int G) {
  if (L == 1) return 0;
  return with_states(N, [&](auto geo) -> size_t {
    const Chunks ck = plan(batch, L, H, N, G, decltype(geo)::CH);
    return ck.count == 1 ? 0 : sizeof(float) * (size_t)batch * ck.count * H * (N + 1) + s4impl::kGap;
  });
}

cudaError_t launch_selective_scan(const s4_selective_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return scan_t<float>(a, st, s);
  if (a.dtype == S4_BF16) return scan_t<__nv_bfloat16>(a, st, s);
  return scan_t<__half>(a, st, s);
}

}  // namespace s4impl
