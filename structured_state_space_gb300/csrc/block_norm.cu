// What joins two blocks, forward and backward: the gate and norm after a block, its residual
// scale, the residual sum and the norm before the next block.
//
//   v = o silu(gate), p = v r1 w_post, h' = h + scale p, y = h' r2 w_pre,
//   r1 = rsqrt(mean v^2 + eps), r2 = rsqrt(mean h'^2 + eps)
//
// About 20 operations per channel on 8 to 14 bytes: the bound is memory.  A row stays in the
// registers of one warp or one CTA from its read to its results, so every array is
// passed over once; both sums of squares are reductions over the group.
//
// Measured: forward 100 us on 16001 rows of 2560 channels in float16 (5.7 TB/s), 135 in fp32 (6.1); backward 132
// us on 16384 rows of 2048 in bfloat16 (5.6 TB/s), 191 in fp32 (5.6); the residual in fp32.  The gradients
// of more than 8192 channels (4 packs of 8 a thread, 8 of 4 in fp32) spill 860 to 970 bytes of registers a thread.
#include "s4_block.cuh"

namespace {
using namespace s4blk;
using s4impl::St;

constexpr int kMaxThreads = 512;  // of the CTA that holds a row

// K sums over the group that holds a row: a warp, or the CTA's warps.  `red` has a slot per warp;
// two sets of them alternate so that one barrier per round is enough.
template <int MAX, int K>
__device__ __forceinline__ void group_sums(float (&v)[K], float (&red)[2][2][32], int& phase) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if constexpr (MAX > 128) {
    constexpr int MOST = MAX / 32;  // warps, a power of two
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, nw = blockDim.x >> 5, from = lane & (MOST - 1);
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[phase][k][wid] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = from < nw ? red[phase][k][from] : 0.f;
#pragma unroll
      for (int o = MOST / 2; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
    phase ^= 1;
  }
}
template <int MAX>
__device__ __forceinline__ float group_sum(float v, float (&red)[2][2][32], int& phase) {
  float s[1] = {v};
  group_sums<MAX, 1>(s, red, phase);
  return s[0];
}

// A pack of parameters as pairs; `with` where there are none.
template <int V>
__device__ __forceinline__ void ld_param(float2 (&v)[V / 2], const float* p, int c, int n, bool vec, float with) {
  if (p) {
    to_pairs<float, V>(ld_pack<float, V>(p + c, n, vec), v);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = make_float2(with, with);
  }
}
__device__ __forceinline__ float both(float2 v) { return v.x + v.y; }
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

// The rows that a group has on their way: with AHEAD, a row's packs are copied into slots of the
// thread's own (two sets of them) while the row before is worked on; else they are read
// when they are needed.  [2][NT][threads] packs of T, then [2][NR][threads] of R.
template <typename T, typename R, int V, int NV, int NT, int NR, bool AHEAD>
struct Rows {
  Pack<T, V>* st;
  Pack<R, V>* sr;
  __device__ __forceinline__ Rows(char* smem)
      : st(reinterpret_cast<Pack<T, V>*>(smem) + threadIdx.x),
        sr(reinterpret_cast<Pack<R, V>*>(smem + 2 * NT * NV * Pack<T, V>::BYTES * blockDim.x) + threadIdx.x) {}
  __device__ __forceinline__ void fetch_t(int stage, int which, int i, const T* p) {
    fetch_whole<T, V>(st + ((stage * NT + which) * NV + i) * blockDim.x, p);
  }
  __device__ __forceinline__ void fetch_r(int stage, int which, int i, const R* p) {
    fetch_whole<R, V>(sr + ((stage * NR + which) * NV + i) * blockDim.x, p);
  }
  __device__ __forceinline__ void get_t(int stage, int which, int i, const T* p, int n, bool vec,
                                        float2 (&v)[V / 2]) const {
    to_pairs<T, V>(AHEAD ? st[((stage * NT + which) * NV + i) * blockDim.x] : ld_pack<T, V>(p, n, vec), v);
  }
  __device__ __forceinline__ void get_r(int stage, int which, int i, const R* p, int n, bool vec,
                                        float2 (&v)[V / 2]) const {
    to_pairs<R, V>(AHEAD ? sr[((stage * NR + which) * NV + i) * blockDim.x] : ld_pack<R, V>(p, n, vec), v);
  }
};

template <typename T, typename R, int V, int NT, int NR>
constexpr int kRowBytes = 2 * (NT * Pack<T, V>::BYTES + NR * Pack<R, V>::BYTES);  // per thread

// NV packs of V channels per thread, pack i at channel (lane + i * width) V.  Groups walk over the
// rows.  What is absent is neutral: a weight of 1, a residual of 0 (without w_post r1 is 1).
template <typename T, typename R, int V, int NV, int MAX, bool AHEAD>
__global__ void __launch_bounds__(MAX, NV == 1 ? 1024 / MAX : 1) block_norm_kernel(s4_block_norm_args a, bool vec) {
  constexpr bool CTA = MAX > 128;  // a row per CTA, or per warp
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) char norm_smem[];
  int phase = 0, stage = 0;
  const int width = CTA ? blockDim.x : 32, lane = CTA ? threadIdx.x : threadIdx.x & 31;
  const int per = CTA ? 1 : blockDim.x >> 5;
  const long long first = (long long)blockIdx.x * per + (CTA ? 0 : threadIdx.x >> 5), step = (long long)gridDim.x * per;
  const float inv = 1.f / (float)a.H;
  Rows<T, R, V, NV, 2, 1, AHEAD> rows(norm_smem);
  const auto fetch = [&](long long row, int stage) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V;
      if (row >= a.rows || c >= a.H) continue;
      rows.fetch_t(stage, 0, i, static_cast<const T*>(a.o) + row * a.o_row + c);
      if (a.gate) rows.fetch_t(stage, 1, i, static_cast<const T*>(a.gate) + row * a.gate_row + c);
      if (a.h) rows.fetch_r(stage, 0, i, static_cast<const R*>(a.h) + row * a.h_row + c);
    }
    fetch_commit();
  };
  if (AHEAD) fetch(first, 0);
  for (long long row = first; row < a.rows; row += step, stage ^= 1) {
    if (AHEAD) {
      fetch(row + step, stage ^ 1);
      fetched_but<1>();
    }
    float2 v[NV][V / 2], hv[NV][V / 2], ss = two(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
#pragma unroll
      for (int j = 0; j < V / 2; ++j) v[i][j] = hv[i][j] = two(0.f);
      if (n <= 0) continue;
      rows.get_t(stage, 0, i, static_cast<const T*>(a.o) + row * a.o_row + c, n, vec, v[i]);
      if (a.h) rows.get_r(stage, 0, i, static_cast<const R*>(a.h) + row * a.h_row + c, n, vec, hv[i]);
      if (a.gate) {
        float2 g[V / 2];
        rows.get_t(stage, 1, i, static_cast<const T*>(a.gate) + row * a.gate_row + c, n, vec, g);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[i][j] = mul2(v[i][j], silu(g[j]));
      }
#pragma unroll
      for (int j = 0; j < V / 2; ++j) ss = fma2(v[i][j], v[i][j], ss);
    }
    float r1 = 1.f;
    if (a.w_post) r1 = rsqrtf(group_sum<MAX>(both(ss), red, phase) * inv + a.eps);
    ss = two(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (n <= 0) continue;
      float2 w[V / 2], sc[V / 2];
      ld_param<V>(w, a.w_post, c, n, vec, 1.f);
      ld_param<V>(sc, a.scale, c, n, vec, 1.f);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        hv[i][j] = fma2(sc[j], mul2(mul2(v[i][j], two(r1)), w[j]), hv[i][j]);
        ss = fma2(hv[i][j], hv[i][j], ss);
      }
      st_pairs<R, V>(static_cast<R*>(a.h_out) + row * a.h_out_row + c, n, vec, hv[i]);
    }
    if (!a.w_pre) continue;
    const float r2 = rsqrtf(group_sum<MAX>(both(ss), red, phase) * inv + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (n <= 0) continue;
      float2 w[V / 2];
      ld_param<V>(w, a.w_pre, c, n, vec, 1.f);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) w[j] = mul2(mul2(hv[i][j], two(r2)), w[j]);
      st_pairs<T, V>(static_cast<T*>(a.y) + row * a.y_row + c, n, vec, w);
    }
  }
}

// Backward, with unit = v r1, unit2 = h' r2, f = dy w_pre, q = scale w_post:
//   dh = dh' + r2 (f - unit2 mean(f unit2)),  dw_pre = sum_rows dy unit2
//   dv = r1 (q dh - unit mean(q dh unit)),  do = dv silu(gate),  dgate = dv o silu'(gate)
//   U = sum_rows dh unit,  dw_post = scale U,  dscale = w_post U
// Three rounds of reductions per row: the mean of v^2; those of h'^2 and f h', which give
// mean(f unit2) = r2 mean(f h'); and the last mean.  (dh being linear in sums that do not need
// r2, the third could go with the second, but where the two terms of dv nearly cancel that
// costs them their last digits.)  A group walks over rows with the two column sums of its
// channels in registers and leaves them as one row of partial sums.
template <typename T, typename R, int V, int NV, int MAX, bool AHEAD>
__global__ void __launch_bounds__(MAX, NV == 1 ? 512 / MAX : 1)
    block_norm_bwd_kernel(s4_block_norm_bwd_args a, bool vec, float* part) {
  constexpr bool CTA = MAX > 128;  // a row per CTA, or per warp
  __shared__ float red[2][2][32];
  extern __shared__ __align__(16) char norm_smem[];
  int phase = 0, stage = 0;
  const int width = CTA ? blockDim.x : 32, lane = CTA ? threadIdx.x : threadIdx.x & 31;
  const int per = CTA ? 1 : blockDim.x >> 5;
  const long long first = (long long)blockIdx.x * per + (CTA ? 0 : threadIdx.x >> 5), step = (long long)gridDim.x * per;
  const float inv = 1.f / (float)a.H;
  const bool with_dy = a.dy && a.w_pre;
  float2 U[NV][V / 2], s_pre[NV][V / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < V / 2; ++j) U[i][j] = s_pre[i][j] = two(0.f);

  Rows<T, R, V, NV, 3, 2, AHEAD> rows(norm_smem);
  const auto fetch = [&](long long row, int stage) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V;
      if (row >= a.rows || c >= a.H) continue;
      rows.fetch_t(stage, 0, i, static_cast<const T*>(a.o) + row * a.o_row + c);
      if (a.gate) rows.fetch_t(stage, 1, i, static_cast<const T*>(a.gate) + row * a.gate_row + c);
      if (with_dy) rows.fetch_t(stage, 2, i, static_cast<const T*>(a.dy) + row * a.dy_row + c);
      if (a.h && with_dy) rows.fetch_r(stage, 0, i, static_cast<const R*>(a.h) + row * a.h_row + c);
      if (a.dh_out) rows.fetch_r(stage, 1, i, static_cast<const R*>(a.dh_out) + row * a.dh_out_row + c);
    }
    fetch_commit();
  };
  if (AHEAD) fetch(first, 0);
  // q and w_pre: with one pack per thread they stay in registers
  float2 q[V / 2], wp[V / 2];
  const auto ld_params = [&](int i) {
    const int c = (lane + i * width) * V, n = a.H - c;
    float2 w[V / 2];
    ld_param<V>(w, a.w_post, c, n, vec, 1.f);
    ld_param<V>(q, a.scale, c, n, vec, 1.f);
    ld_param<V>(wp, a.w_pre, c, n, vec, 1.f);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) q[j] = mul2(q[j], w[j]);
  };
  if (NV == 1) ld_params(0);
  for (long long row = first; row < a.rows; row += step, stage ^= 1) {
    const T* o = static_cast<const T*>(a.o) + row * a.o_row;
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + row * a.gate_row : nullptr;
    if (AHEAD) {
      fetch(row + step, stage ^ 1);
      fetched_but<1>();
    }
    float2 v[NV][V / 2], hv[NV][V / 2], d[NV][V / 2], ss = two(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
#pragma unroll
      for (int j = 0; j < V / 2; ++j) v[i][j] = hv[i][j] = d[i][j] = two(0.f);
      if (n <= 0) continue;
      rows.get_t(stage, 0, i, o + c, n, vec, v[i]);
      if (with_dy) {
        rows.get_t(stage, 2, i, static_cast<const T*>(a.dy) + row * a.dy_row + c, n, vec, d[i]);
        if (a.h) rows.get_r(stage, 0, i, static_cast<const R*>(a.h) + row * a.h_row + c, n, vec, hv[i]);
      }
      if (gate) {
        float2 g[V / 2];
        rows.get_t(stage, 1, i, gate + c, n, vec, g);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[i][j] = mul2(v[i][j], silu(g[j]));
      }
#pragma unroll
      for (int j = 0; j < V / 2; ++j) ss = fma2(v[i][j], v[i][j], ss);
    }
    float r1 = 1.f;
    if (a.w_post) r1 = rsqrtf(group_sum<MAX>(both(ss), red, phase) * inv + a.eps);
    // v -> unit; h'
    float r2 = 0.f, m2 = 0.f;
    if (with_dy) {
      float2 s0 = two(0.f), s1 = two(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (lane + i * width) * V, n = a.H - c;
        if (n <= 0) continue;
        if (NV > 1) ld_params(i);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          v[i][j] = mul2(v[i][j], two(r1));
          hv[i][j] = fma2(q[j], v[i][j], hv[i][j]);
          s0 = fma2(hv[i][j], hv[i][j], s0);
          s1 = fma2(mul2(d[i][j], wp[j]), hv[i][j], s1);
        }
      }
      float sum[2] = {both(s0), both(s1)};
      group_sums<MAX, 2>(sum, red, phase);
      r2 = rsqrtf(sum[0] * inv + a.eps);
      m2 = r2 * sum[1] * inv;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V / 2; ++j) v[i][j] = mul2(v[i][j], two(r1));
    }
    // d -> dh, then q dh
    ss = two(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (n <= 0) continue;
      float2 e[V / 2];
      if (NV > 1) ld_params(i);
      if (a.dh_out)
        rows.get_r(stage, 1, i, static_cast<const R*>(a.dh_out) + row * a.dh_out_row + c, n, vec, e);
      else
#pragma unroll
        for (int j = 0; j < V / 2; ++j) e[j] = two(0.f);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 unit2 = mul2(hv[i][j], two(r2));
        s_pre[i][j] = fma2(d[i][j], unit2, s_pre[i][j]);
        e[j] = fma2(two(r2), fma2(unit2, two(-m2), mul2(d[i][j], wp[j])), e[j]);
        U[i][j] = fma2(e[j], v[i][j], U[i][j]);
        d[i][j] = mul2(e[j], q[j]);
        ss = fma2(d[i][j], v[i][j], ss);
      }
      if (a.dh) st_pairs<R, V>(static_cast<R*>(a.dh) + row * a.dh_row + c, n, vec, e);
    }
    const float m1 = a.w_post ? group_sum<MAX>(both(ss), red, phase) * inv : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (lane + i * width) * V, n = a.H - c;
      if (n <= 0) continue;
#pragma unroll
      for (int j = 0; j < V / 2; ++j) d[i][j] = mul2(two(r1), fma2(v[i][j], two(-m1), d[i][j]));
      if (gate) {
        float2 g[V / 2], ov[V / 2];
        rows.get_t(stage, 1, i, gate + c, n, vec, g);
        rows.get_t(stage, 0, i, o + c, n, vec, ov);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
          const float2 s = sigmoid(g[j]), act = mul2(g[j], s);
          ov[j] = mul2(mul2(ov[j], d[i][j]), fma2(act, fma2(s, two(-1.f), two(1.f)), s));
          d[i][j] = mul2(d[i][j], act);
        }
        st_pairs<T, V>(static_cast<T*>(a.dgate) + row * a.dgate_row + c, n, vec, ov);
      }
      st_pairs<T, V>(static_cast<T*>(a.do_) + row * a.do_row + c, n, vec, d[i]);
    }
  }
  // part[group][2][H]
  float* out = part + first * 2 * a.H;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (lane + i * width) * V;
    if (a.H - c <= 0) continue;
    st_pairs<float, V>(out + c, a.H - c, a.H % 4 == 0, U[i]);
    st_pairs<float, V>(out + a.H + c, a.H - c, a.H % 4 == 0, s_pre[i]);
  }
}

__global__ void __launch_bounds__(256) block_norm_sums_kernel(const float* part, int rows, s4_block_norm_bwd_args a) {
  column_sums(part, rows, 2ll * a.H, 2ll * a.H, [=](long long c, float v) {
    const int h = (int)(c % a.H);
    if (c >= a.H) {
      if (a.dw_pre) wr(a.dw_pre + h, v);
    } else {
      if (a.dw_post) wr(a.dw_post + h, a.scale ? rd(a.scale + h) * v : v);
      if (a.dscale) wr(a.dscale + h, a.w_post ? rd(a.w_post + h) * v : v);
    }
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
// CTAs that walk over rows read ahead: as many as run at once (asked once per device, kernel and
// CTA size; a grid of 1.5 rounds took 142 us instead of 102 forward on 16001 rows of 2560 channels).
// Rows that are not read ahead have a group each in the forward pass.  In the backward pass each
// group leaves one row of partial sums, of kMostThreads threads per SM at most.
constexpr int kMaxAhead = 200 * 1024, kMostThreads = 1024;
int most_ctas(long long rows, const Shape& sh, int per_sm) {
  const long long per = sh.cta ? 1 : sh.threads / 32, need = (rows + per - 1) / per;
  const int fit = kMostThreads / sh.threads < per_sm ? kMostThreads / sh.threads : per_sm;
  const long long most = (long long)s4impl::num_sms() * (fit < 1 ? 1 : fit);
  return (int)(need < most ? need : most);
}
template <auto Kernel>
int ctas_for(long long rows, const Shape& sh, int bytes) {
  static std::atomic<int> known[64][kMaxThreads / 32 + 1];
  allow_shared<Kernel>(kMaxAhead);
  std::atomic<int>& k = known[device()][sh.threads / 32];
  int per_sm = k.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, Kernel, sh.threads, bytes) != cudaSuccess || per_sm < 1)
      per_sm = 1;
    k.store(per_sm, std::memory_order_relaxed);
  }
  return most_ctas(rows, sh, per_sm);
}

// f(kernel shape as constants: packs per thread, largest CTA)
template <int V, typename F>
void with_shape(const Shape& sh, F f) {
  if (!sh.cta) {
    if (sh.nv == 1) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 128>{});
    return f(std::integral_constant<int, 2>{}, std::integral_constant<int, 128>{});
  }
  if (sh.nv == 1 && sh.threads <= 256) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, 256>{});
  if (sh.nv == 1) return f(std::integral_constant<int, 1>{}, std::integral_constant<int, kMaxThreads>{});
  if (sh.nv == 2) return f(std::integral_constant<int, 2>{}, std::integral_constant<int, kMaxThreads>{});
  if (sh.nv == 4) return f(std::integral_constant<int, 4>{}, std::integral_constant<int, kMaxThreads>{});
  if constexpr (V == 4)  // 16384 channels in 32 bits
    return f(std::integral_constant<int, 8>{}, std::integral_constant<int, kMaxThreads>{});
}

template <typename T, typename R, int V>
cudaError_t fwd_t(const s4_block_norm_args& a, cudaStream_t s) {
  const int et = sizeof(T), er = sizeof(R), bt = sizeof(Pack<T, V>), br = sizeof(Pack<R, V>);
  const bool vec = vec_ok(a.o, et, bt, a.o_row) && vec_ok(a.gate, et, bt, a.gate_row) &&
                   vec_ok(a.h, er, br < 16 ? br : 16, a.h_row) && vec_ok(a.h_out, er, br < 16 ? br : 16, a.h_out_row) &&
                   vec_ok(a.y, et, bt, a.y_row) && vec_ok(a.w_post, 4, 16) && vec_ok(a.scale, 4, 16) &&
                   vec_ok(a.w_pre, 4, 16);
  const Shape sh = shape_for(a.H, V);
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.add(a.o, et, true, false, a.H, a.rows, a.o_row);
  x.add(a.gate, et, true, false, a.H, a.rows, a.gate_row);
  x.add(a.h, er, true, false, a.H, a.rows, a.h_row);
  x.add(a.h_out, er, false, true, a.H, a.rows, a.h_out_row);
  x.add(a.y, et, false, true, a.H, a.rows, a.y_row);
  for (const float* p : {a.w_post, a.scale, a.w_pre}) x.in(p, 4, a.H);
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  s4impl::TimedLaunch tl("block_norm", s);
  with_shape<V>(sh, [&](auto nv, auto max) {
    constexpr int NV = decltype(nv)::value, MAX = decltype(max)::value;
    if constexpr (NV <= 2) {
      const int bytes = NV * kRowBytes<T, R, V, 2, 1> * sh.threads;
      if (vec && a.H % V == 0 && bytes <= kMaxAhead) {
        constexpr auto kernel = block_norm_kernel<T, R, V, NV, MAX, true>;
        kernel<<<ctas_for<kernel>(a.rows, sh, bytes), sh.threads, bytes, s>>>(a, vec);
        return;
      }
    }
    const long long per = sh.cta ? 1 : sh.threads / 32;
    block_norm_kernel<T, R, V, NV, MAX, false><<<(unsigned)((a.rows + per - 1) / per), sh.threads, 0, s>>>(a, vec);
  });
  return cudaGetLastError();
}

template <typename T, typename R, int V>
cudaError_t bwd_t(const s4_block_norm_bwd_args& a, cudaStream_t s) {
  const int et = sizeof(T), er = sizeof(R), bt = sizeof(Pack<T, V>), br = sizeof(Pack<R, V>) < 16 ? sizeof(Pack<R, V>) : 16;
  const bool vec = vec_ok(a.o, et, bt, a.o_row) && vec_ok(a.gate, et, bt, a.gate_row) && vec_ok(a.h, er, br, a.h_row) &&
                   vec_ok(a.dy, et, bt, a.dy_row) && vec_ok(a.dh_out, er, br, a.dh_out_row) &&
                   vec_ok(a.do_, et, bt, a.do_row) && vec_ok(a.dgate, et, bt, a.dgate_row) &&
                   vec_ok(a.dh, er, br, a.dh_row) && vec_ok(a.w_post, 4, 16) && vec_ok(a.scale, 4, 16) &&
                   vec_ok(a.w_pre, 4, 16);
  const Shape sh = shape_for(a.H, V);
  int grid = 0;
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + s4impl::kStatusBytes);
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.add(a.o, et, true, false, a.H, a.rows, a.o_row);
  x.add(a.gate, et, true, false, a.H, a.rows, a.gate_row);
  x.add(a.h, er, true, false, a.H, a.rows, a.h_row);
  x.add(a.dy, et, true, false, a.H, a.rows, a.dy_row);
  x.add(a.dh_out, er, true, false, a.H, a.rows, a.dh_out_row);
  x.add(a.do_, et, false, true, a.H, a.rows, a.do_row);
  x.add(a.dgate, et, false, true, a.H, a.rows, a.dgate_row);
  x.add(a.dh, er, false, true, a.H, a.rows, a.dh_row);
  for (const float* p : {a.w_post, a.scale, a.w_pre}) x.in(p, 4, a.H);
  for (const float* p : {a.dw_post, a.dscale, a.dw_pre}) x.out(p, 4, a.H);
  x.scratch(part, 4, a.H, (long long)(s4impl::block_norm_bwd_scratch(a.rows, a.H) / (4ull * a.H)));
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  {
    s4impl::TimedLaunch tl("block_norm_bwd", s);
    with_shape<V>(sh, [&](auto nv, auto max) {
      constexpr int NV = decltype(nv)::value, MAX = decltype(max)::value;
      if constexpr (NV <= 2) {
        const int bytes = NV * kRowBytes<T, R, V, 3, 2> * sh.threads;
        if (vec && a.H % V == 0 && bytes <= kMaxAhead) {
          constexpr auto kernel = block_norm_bwd_kernel<T, R, V, NV, MAX, true>;
          grid = ctas_for<kernel>(a.rows, sh, bytes);
          kernel<<<grid, sh.threads, bytes, s>>>(a, vec, part);
          return;
        }
      }
      constexpr auto kernel = block_norm_bwd_kernel<T, R, V, NV, MAX, false>;
      grid = ctas_for<kernel>(a.rows, sh, 0);
      kernel<<<grid, sh.threads, 0, s>>>(a, vec, part);
    });
  }
  if (!a.dw_post && !a.dscale && !a.dw_pre) return cudaGetLastError();
  s4impl::TimedLaunch tl("block_norm_bwd", s);
  block_norm_sums_kernel<<<(unsigned)((2ll * a.H + 31) / 32), 256, 0, s>>>(part, grid * (sh.cta ? 1 : sh.threads / 32), a);
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
    const size_t r = (size_t)most_ctas(rows, sh, 16) * (sh.cta ? 1 : sh.threads / 32);
    most = r > most ? r : most;
  }
  return sizeof(float) * 2 * most * (size_t)H;
}

cudaError_t launch_block_norm_bwd(const s4_block_norm_bwd_args& a, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float, float, 4>(a, s);
  if (a.dtype == S4_BF16)
    return a.res_f32 ? bwd_t<__nv_bfloat16, float, 8>(a, s) : bwd_t<__nv_bfloat16, __nv_bfloat16, 8>(a, s);
  return a.res_f32 ? bwd_t<__half, float, 8>(a, s) : bwd_t<__half, __half, 8>(a, s);
}

}  // namespace s4impl
