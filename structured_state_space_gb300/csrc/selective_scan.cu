// The selective state-space scan, forward: prompts and single tokens.
//
//   d = softplus(dt + dt_bias),  s_n = 2^(d A_n log2 e) s_n + d x B_n,  y = (sum_n C_n s_n + D x) silu(z)
//
// Per (token, channel, state): one exponential (the SM's special function units give 32 of them
// a clock) and four multiplications or additions (128 a clock), so that both pipes need 4
// clocks of an SM quarter for 32 of them; the activations are 8 bytes per (token, channel) in
// 16 bits.  At N = 16 the exponentials bound it, not memory.
//
// The recurrence is sequential in time, parallel over sequences, channels and states.  A CTA
// takes HB channels and walks a stretch of tokens, in tiles of TT tokens staged in shared
// memory: the step sizes and inputs are formed once per (token, channel) there, and read by
// the LPC lanes that share the channel.  Where there are too few channels to fill the GPU, the
// tokens are split into chunks: a first kernel gives each chunk's state from a zero start
// and its total step (which fixes its decay), a second joins them, the third runs the chunks
// from their true starts.  That costs the exponentials twice.
#include "selective.cuh"

namespace {
using namespace s4sel;

template <int LPC_, int SPT_>
struct Geo {
  static constexpr int LPC = LPC_, SPT = SPT_, NP = LPC * SPT;
  static constexpr int HB = 2 * kThreads / LPC;      // channels of a CTA
  static constexpr int TT = 16;                      // tokens of a tile
  static constexpr int CELLS = TT * HB / kThreads;   // (token, channel) cells a thread stages
  static constexpr int VECS = TT * NP / kThreads;    // and elements of B, of C
  // Shared memory in floats: step and step x of channel pairs [TT][HB / 2][4] | B and C, each
  // element twice (for both halves of a pair) [TT][NP][2] | y [TT][YROW].  The rows of y are 8
  // floats longer than HB: the 4 tokens and 8 channel pairs a warp writes lie in different banks.
  static constexpr int YROW = HB + 8;
  static constexpr int B0 = 2 * TT * HB, C0 = B0 + 2 * TT * NP, Y0 = C0 + 2 * TT * NP;
  static constexpr int bytes(int mode) { return 4 * (mode ? Y0 + TT * YROW : C0); }
};

struct Chunks {
  int len, count;   // tokens per chunk (a multiple of the tile), number of chunks
  float *start;     // [batch][count][H][N]: end states from zero, then start states
  float *total;     // [batch][count][H]: sums of the step sizes
};

// V consecutive elements per access, of `count` a thread takes.
template <typename T>
constexpr int pack_of(int count, int row) {
  int v = 16 / (int)sizeof(T);
  v = v < row ? v : row;
  return v < count ? v : count;
}

// MODE 0: states from a zero start and total steps of chunks 0 .. count - 2; MODE 1: outputs.
// A tile's global reads are issued before the tile ahead of it is computed and wait in
// registers until that is done.
template <typename T, typename G, int MODE>
__global__ void __launch_bounds__(kThreads) selective_scan_kernel(s4_selective_args a, Chunks ck, bool vec, bool vecbc,
                                                                 St st) {
  constexpr int LPC = G::LPC, SPT = G::SPT, NP = G::NP, HB = G::HB, TT = G::TT;
  constexpr int V = pack_of<T>(G::CELLS, HB), NV = G::CELLS / V, STEP = kThreads * V / HB;  // tokens between packs
  constexpr int VB = pack_of<T>(G::VECS, NP), NB = G::VECS / VB;
  extern __shared__ __align__(16) float smem[];
  float4(*sd)[HB / 2] = reinterpret_cast<float4(*)[HB / 2]>(smem);
  float2(*sb)[NP] = reinterpret_cast<float2(*)[NP]>(smem + G::B0);
  float2(*sc)[NP] = reinterpret_cast<float2(*)[NP]>(smem + G::C0);
  float(*sy)[G::YROW] = reinterpret_cast<float(*)[G::YROW]>(smem + G::Y0);
  record_gen(st);
  const int b = blockIdx.z, chunk = blockIdx.y;
  const Chan c = chan_of<HB>(blockIdx.x, a.H / a.G);
  const Seq q = seq_of(a.lengths, a.index, b, a.L, a.slots, st);
  const int t0 = chunk * ck.len, t1 = min(a.L, t0 + ck.len), live = min(t1, q.len);
  if (MODE == 0 && t0 >= q.len) return;
  const int lane = threadIdx.x % LPC, slot = threadIdx.x / LPC, n0 = lane * SPT;
  // the cells this thread stages: channels h .. h + V of tokens row, row + STEP, ...
  const int hl = threadIdx.x * V % HB, row = threadIdx.x * V / HB, h = c.h0 + hl, nh = c.hend - h;
  const T* x = static_cast<const T*>(a.x.p) + b * a.x.batch + h;
  const T* dt = static_cast<const T*>(a.dt.p) + b * a.dt.batch + h;
  const T* z = MODE && a.z.p ? static_cast<const T*>(a.z.p) + b * a.z.batch + h : nullptr;
  const T* B = static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group;
  const T* C = static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group;
  T* y = MODE ? static_cast<T*>(a.y.p) + b * a.y.batch + h : nullptr;
  float bias[V], skip[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = a.dt_bias && i < nh ? a.dt_bias[h + i] : 0.f;
    skip[i] = MODE && a.D && i < nh ? a.D[h + i] : 0.f;
  }

  float2 A[SPT], s[SPT], sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < SPT; ++i) {
    float Av[2], sv[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int hs = c.h0 + 2 * slot + j, n = n0 + i;
      const bool in = hs < c.hend && n < a.N;
      Av[j] = in ? a.A[(long long)hs * a.N + n] * kLog2e : 0.f;
      sv[j] = 0.f;
      if (MODE == 1 && in && (t0 < q.len || chunk == 0)) {
        if (ck.count > 1)
          sv[j] = ck.start[(((long long)b * ck.count + chunk) * a.H + hs) * a.N + n];
        else if (a.state && q.slot >= 0)
          sv[j] = a.state[(q.slot * a.H + hs) * a.N + n];
      }
    }
    A[i] = make_float2(Av[0], Av[1]);
    s[i] = make_float2(sv[0], sv[1]);
  }

  Pack<T, V> px[NV], pz[NV], nx[NV], nz[NV], nd[NV];
  Pack<T, VB> nb[NB], nc[NB];
  const auto fetch = [&](int tb) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int t = tb + row + k * STEP;
      const int n = t < live && S4_IN(t, a.L) ? nh : 0;
      nx[k] = ld_pack<T, V>(x + t * a.x.row, n, vec);
      nd[k] = ld_pack<T, V>(dt + t * a.dt.row, n, vec);
      if (z) nz[k] = ld_pack<T, V>(z + t * a.z.row, n, vec);
    }
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      const int i = (k * kThreads + threadIdx.x) * VB, t = tb + i / NP;
      const int n = t < live && S4_IN(t, a.L) ? a.N - i % NP : 0;
      nb[k] = ld_pack<T, VB>(B + t * a.B.row + i % NP, n, vecbc);
      if (MODE == 1) nc[k] = ld_pack<T, VB>(C + t * a.C.row + i % NP, n, vecbc);
    }
  };
  if (t0 < live) fetch(t0);
  for (int tb = t0; tb < (MODE ? t1 : live); tb += TT) {
    if (tb < live) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        px[k] = nx[k];
        pz[k] = nz[k];
        float d[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          d[i] = nd[k].get(i) + bias[i];
          if (a.softplus) d[i] = softplus(d[i]);
          if (tb + row + k * STEP >= live || i >= nh) d[i] = 0.f;
        }
        float* to = reinterpret_cast<float*>(&sd[row + k * STEP][0]) + 2 * hl;
        if constexpr (V == 1) {
          // (step, step x) of one half of a pair
          to = reinterpret_cast<float*>(&sd[row + k * STEP][hl / 2]) + hl % 2;
          to[0] = d[0];
          to[2] = d[0] * px[k].get(0);
        } else {
#pragma unroll
          for (int i = 0; i < V; i += 2)
            *reinterpret_cast<float4*>(to + 2 * i) =
                make_float4(d[i], d[i + 1], d[i] * px[k].get(i), d[i + 1] * px[k].get(i + 1));
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int i = (k * kThreads + threadIdx.x) * VB;
#pragma unroll
        for (int e = 0; e < VB; ++e) {
          const float vb = nb[k].get(e);
          (&sb[0][0])[i + e] = make_float2(vb, vb);
          if (MODE == 1) {
            const float vc = nc[k].get(e);
            (&sc[0][0])[i + e] = make_float2(vc, vc);
          }
        }
      }
      __syncthreads();
      if (tb + TT < live) fetch(tb + TT);
#pragma unroll
      for (int u = 0; u < TT; u += 4) {
        float2 v[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float4 d = sd[u + w][slot];
          const float2 dd = make_float2(d.x, d.y), dx = make_float2(d.z, d.w);
          if (MODE == 0) sum = add2(sum, dd);
#pragma unroll
          for (int i = 0; i < SPT; i += 2) {
            const float4 b4 = *reinterpret_cast<const float4*>(&sb[u + w][n0 + i]);
            s[i] = fma2(ex2(mul2(dd, A[i])), s[i], mul2(dx, make_float2(b4.x, b4.y)));
            s[i + 1] = fma2(ex2(mul2(dd, A[i + 1])), s[i + 1], mul2(dx, make_float2(b4.z, b4.w)));
            if (MODE == 1) {
              const float4 c4 = *reinterpret_cast<const float4*>(&sc[u + w][n0 + i]);
              v[w] = i ? fma2(make_float2(c4.x, c4.y), s[i], v[w]) : mul2(make_float2(c4.x, c4.y), s[i]);
              v[w] = fma2(make_float2(c4.z, c4.w), s[i + 1], v[w]);
            }
          }
        }
        if (MODE == 1) {
          sum_lanes<LPC>(v, lane);
          if (lane < 4) {
#pragma unroll
            for (int i = 0; i < kOwn<LPC>; ++i)
              *reinterpret_cast<float2*>(&sy[u + own_token<LPC>(lane, i)][2 * slot]) = v[i];
          }
        }
      }
      __syncthreads();
    }
    if (MODE == 1) {
      // the outputs of this thread's cells: skip term, gate, one rounding
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int t = tb + row + k * STEP;
        if (t >= t1 || nh <= 0 || !S4_IN(t, a.L)) continue;
        float out[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
          out[i] = 0.f;
          if (t < live) {
            const float v = fmaf(skip[i], px[k].get(i), sy[row + k * STEP][hl + i]);
            out[i] = z ? v * silu(pz[k].get(i)) : v;
          }
        }
        st_f<T, V>(y + t * a.y.row, nh, vec, out);
      }
    }
  }
  // Where the state goes: the chunk's end state, or, after the last real token, the caller's slot.
  float* out = nullptr;
  if (MODE == 0)
    out = ck.start + ((long long)b * ck.count + chunk) * a.H * a.N;
  else if (a.state_out && q.slot >= 0 && ((t0 < q.len && q.len <= t1) || (q.len == 0 && chunk == 0)) &&
           S4_IN(q.slot, a.slots))
    out = a.state_out + q.slot * a.H * a.N;
  if (out) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int hs = c.h0 + 2 * slot + j;
      if (hs >= c.hend) continue;
#pragma unroll
      for (int i = 0; i < SPT; ++i)
        if (n0 + i < a.N) out[(long long)hs * a.N + n0 + i] = j ? s[i].y : s[i].x;
      if (MODE == 0 && lane == 0) ck.total[((long long)b * ck.count + chunk) * a.H + hs] = j ? sum.y : sum.x;
    }
  }
}

// Joins the chunks: start_{c+1} = 2^(A total_c) start_c + end_c, in place of the end states.
__global__ void __launch_bounds__(256) selective_join_kernel(s4_selective_args a, Chunks ck, St st) {
  const int b = blockIdx.y;
  const Seq q = seq_of(a.lengths, a.index, b, a.L, a.slots, st);
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, HN = (long long)a.H * a.N;
  if (i >= HN) return;
  const int h = (int)(i / a.N);
  const float A = a.A[i] * kLog2e;
  float s = a.state && q.slot >= 0 ? a.state[q.slot * HN + i] : 0.f;
  for (int c = 0; c < ck.count && (c == 0 || c * ck.len < q.len); ++c) {
    float* p = ck.start + ((long long)b * ck.count + c) * HN + i;
    const bool more = c + 1 < ck.count && (c + 1) * ck.len < q.len;
    const float end = more ? *p : 0.f, d = more ? ck.total[((long long)b * ck.count + c) * a.H + h] : 0.f;
    *p = s;
    s = fmaf(ex2(d * A), s, end);
  }
}

// One token per sequence: the state is read, advanced and written once (8 bytes per channel and
// state, which bound it).
template <typename T, int LPC, int SPT>
__global__ void __launch_bounds__(256) selective_step_kernel(s4_selective_args a, bool vec, St st) {
  constexpr int HB = 256 / LPC;
  record_gen(st);
  const int b = blockIdx.y;
  const Chan c = chan_of<HB>(blockIdx.x, a.H / a.G);
  const Seq q = seq_of(a.lengths, a.index, b, 1, a.slots, st);
  const int lane = threadIdx.x % LPC, h = c.h0 + threadIdx.x / LPC, n0 = lane * SPT, n = a.N - n0;
  float acc = 0.f, xv = 0.f, zv = 0.f;
  if (h < c.hend && q.slot >= 0) {
    const long long at = (q.slot * a.H + h) * a.N + n0;
    float s[SPT];
#pragma unroll
    for (int i = 0; i < SPT; ++i) s[i] = 0.f;
    if (n > 0 && a.state && S4_IN(q.slot, a.slots))
      ld_f<float, SPT>(a.state + at, n, vec, s);
    if (q.len > 0) {
      float A[SPT], Bv[SPT], Cv[SPT];
      xv = to_f(static_cast<const T*>(a.x.p)[b * a.x.batch + h]);
      float d = to_f(static_cast<const T*>(a.dt.p)[b * a.dt.batch + h]);
      if (a.z.p) zv = to_f(static_cast<const T*>(a.z.p)[b * a.z.batch + h]);
      if (a.dt_bias) d += a.dt_bias[h];
      if (a.softplus) d = softplus(d);
      if (n > 0) {
        ld_f<float, SPT>(a.A + (long long)h * a.N + n0, n, vec, A);
        ld_f<T, SPT>(static_cast<const T*>(a.B.p) + b * a.B.batch + c.g * a.B_group + n0, n, false, Bv);
        ld_f<T, SPT>(static_cast<const T*>(a.C.p) + b * a.C.batch + c.g * a.C_group + n0, n, false, Cv);
#pragma unroll
        for (int i = 0; i < SPT; ++i) {
          s[i] = fmaf(ex2(d * A[i] * kLog2e), s[i], d * xv * Bv[i]);
          acc = fmaf(Cv[i], s[i], acc);
        }
      }
    }
    if (n > 0 && a.state_out && S4_IN(q.slot, a.slots)) st_f<float, SPT>(a.state_out + at, n, vec, s);
  }
#pragma unroll
  for (int o = LPC / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0 && h < c.hend) {
    if (a.D && q.len > 0) acc = fmaf(a.D[h], xv, acc);
    if (a.z.p) acc *= silu(zv);
    static_cast<T*>(a.y.p)[b * a.y.batch + h] = from_f<T>(q.len > 0 ? acc : 0.f);
  }
}

// Chunks: enough warps to fill the GPU (kWarps per SM), none shorter than kMinChunk tokens, and
// only where one chunk would leave more than half of them missing (chunks read the inputs twice).
constexpr int kWarps = 16, kMinChunk = 128, kTile = 16;
Chunks plan(int batch, int L, int H, int N, int G, int HB) {
  const long long ctas = (long long)batch * G * ((H / G + HB - 1) / HB);
  const long long want = (long long)s4impl::num_sms() * kWarps / (kThreads / 32);
  Chunks ck{L, 1, nullptr, nullptr};
  if (2 * ctas > want || L < 2 * kMinChunk) return ck;
  long long n = (want + ctas - 1) / ctas;
  if (n > L / kMinChunk) n = L / kMinChunk;
  ck.len = (int)(((L + n - 1) / n + kTile - 1) / kTile * kTile);
  ck.count = (L + ck.len - 1) / ck.len;
  return ck;
}

// The lanes and states per lane that hold N states.
template <typename F>
auto with_states(int N, F f) {
  if (N <= 8) return f(Geo<2, 4>{});
  if (N <= 16) return f(Geo<4, 4>{});
  if (N <= 32) return f(Geo<8, 4>{});
  if (N <= 64) return f(Geo<16, 4>{});
  if (N <= 128) return f(Geo<32, 4>{});
  return f(Geo<32, 8>{});
}

template <typename T>
cudaError_t step_t(const s4_selective_args& a, St st, cudaStream_t s) {
  const bool vec = a.N % 4 == 0 && vec_ok(a.state, 4, 16) && vec_ok(a.state_out, 4, 16) && vec_ok(a.A, 4, 16);
  s4impl::TimedLaunch tl("selective_step", s);
  with_states(a.N, [&](auto geo) {
    using G = decltype(geo);
    constexpr int HB = 256 / G::LPC;
    const dim3 grid(a.G * ((a.H / a.G + HB - 1) / HB), a.batch);
    selective_step_kernel<T, G::LPC, G::SPT><<<grid, 256, 0, s>>>(a, vec, st);
  });
  return cudaGetLastError();
}

template <typename T>
cudaError_t scan_t(const s4_selective_args& a, St st, cudaStream_t s) {
  if (a.L == 1) return step_t<T>(a, st, s);
  const int e = sizeof(T);
  with_states(a.N, [&](auto geo) {
    using G = decltype(geo);
    const bool vec = vec_ok(a.x.p, e, 16, a.x.batch, a.x.row) && vec_ok(a.dt.p, e, 16, a.dt.batch, a.dt.row) &&
                     vec_ok(a.z.p, e, 16, a.z.batch, a.z.row) && vec_ok(a.y.p, e, 16, a.y.batch, a.y.row) &&
                     (a.G == 1 || (a.H / a.G) * e % 16 == 0);
    constexpr int pb = sizeof(T) * pack_of<T>(G::VECS, G::NP);
    const bool vecbc = vec_ok(a.B.p, e, pb, a.B.batch, a.B.row) && vec_ok(a.C.p, e, pb, a.C.batch, a.C.row) &&
                       a.B_group * e % pb == 0 && a.C_group * e % pb == 0;
    Chunks ck = plan(a.batch, a.L, a.H, a.N, a.G, G::HB);
    ck.start = reinterpret_cast<float*>(static_cast<char*>(a.ws) + s4impl::kStatusBytes);
    ck.total = ck.start + (long long)a.batch * ck.count * a.H * a.N;
    const int blocks = a.G * ((a.H / a.G + G::HB - 1) / G::HB);
    for (auto k : {selective_scan_kernel<T, G, 0>, selective_scan_kernel<T, G, 1>})
      if (G::bytes(1) > 48 * 1024) cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, G::bytes(1));
    if (ck.count > 1) {
      {
        s4impl::TimedLaunch tl("selective_scan", s);
        selective_scan_kernel<T, G, 0>
            <<<dim3(blocks, ck.count - 1, a.batch), kThreads, G::bytes(0), s>>>(a, ck, vec, vecbc, st);
      }
      s4impl::TimedLaunch tl("selective_scan", s);
      const long long HN = (long long)a.H * a.N;
      selective_join_kernel<<<dim3((unsigned)((HN + 255) / 256), a.batch), 256, 0, s>>>(a, ck, st);
    }
    s4impl::TimedLaunch tl("selective_scan", s);
    selective_scan_kernel<T, G, 1><<<dim3(blocks, ck.count, a.batch), kThreads, G::bytes(1), s>>>(a, ck, vec, vecbc, st);
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
    const Chunks ck = plan(batch, L, H, N, G, decltype(geo)::HB);
    return ck.count == 1 ? 0 : sizeof(float) * (size_t)batch * ck.count * H * (N + 1);
  });
}

cudaError_t launch_selective_scan(const s4_selective_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return scan_t<float>(a, st, s);
  if (a.dtype == S4_BF16) return scan_t<__nv_bfloat16>(a, st, s);
  return scan_t<__half>(a, st, s);
}

}  // namespace s4impl
