// Rows of channels held in the registers of one warp or one CTA, from their read to their results:
// reductions over the group, rows read ahead through shared memory, launch shapes.  Shared by the
// block norms and the layer norm.
#pragma once
#include "s4_block.cuh"

namespace {
using namespace s4blk;

constexpr int kMaxThreads = 512;  // of the CTA that holds a row

// K sums over the group that holds a row: a warp, or the CTA's warps.  `red` has a slot per warp;
// two sets of them alternate so that one barrier per round is enough.
template <int MAX, int K, int KR>
__device__ __forceinline__ void group_sums(float (&v)[K], float (&red)[2][KR][32], int& phase) {
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
template <typename T, typename R, int V, int NV, int NT, int NR, bool AHEAD, int SETS = 2>
struct Rows {
  Pack<T, V>* st;
  Pack<R, V>* sr;
  __device__ __forceinline__ Rows(char* smem)
      : st(reinterpret_cast<Pack<T, V>*>(smem) + threadIdx.x),
        sr(reinterpret_cast<Pack<R, V>*>(smem + SETS * NT * NV * Pack<T, V>::BYTES * blockDim.x) + threadIdx.x) {}
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

template <typename T, typename R, int V, int NT, int NR, int SETS = 2>
constexpr int kRowBytes = SETS * (NT * Pack<T, V>::BYTES + NR * Pack<R, V>::BYTES);  // per thread

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

}  // namespace
