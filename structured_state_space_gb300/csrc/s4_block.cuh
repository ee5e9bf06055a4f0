// Device building blocks of the selective block's kernels: element types, row
// accesses of one to sixteen bytes, activations, column sums.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "s4_block.h"
#include "s4_dev.cuh"
#include "s4_extents.h"

namespace s4blk {

using s4impl::St;

// ---- accesses to global memory ------------------------------------------------------------------
// touch(): whether an access may be made.  In the bounds-checked build each one is compared with the
// extents of the call's arrays and its address with the access's width; one that does not fit is
// counted and left out (a load gives zero).
#ifdef S4_BOUNDS_CHECK
static __device__ s4impl::Extents g_extents;
static __device__ __noinline__ bool touch(const void* p, int bytes, int align, bool write) {
  const bool ok = s4impl::access_ok(g_extents.list, g_extents.n, reinterpret_cast<unsigned long long>(p), bytes, align, write);
  if (!ok) s4dev::s4_oob_hit();
  return ok;
}
inline cudaError_t set_extents(const s4impl::Extents& x, cudaStream_t s) {
  return cudaMemcpyToSymbolAsync(g_extents, &x, sizeof(x), 0, cudaMemcpyHostToDevice, s);
}
#else
__device__ __forceinline__ constexpr bool touch(const void*, int, int, bool) { return true; }
#endif
template <typename T>
__device__ __forceinline__ T rd(const T* p) {
  return touch(p, sizeof(T), sizeof(T), false) ? *p : T{};
}
template <typename T>
__device__ __forceinline__ void wr(T* p, T v) {
  if (touch(p, sizeof(T), sizeof(T), true)) *p = v;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// V elements of T as they lie in memory, in words of 32 bits (16 where a pack is one 16-bit
// element): a load can then be waited for where its values are used, which packs of separate
// 16-bit values, taken apart where the load's branches meet, do not allow.
template <typename T>
__device__ __forceinline__ unsigned bits_of(T v) {
  if constexpr (sizeof(T) == 4)
    return __float_as_uint(v);
  else
    return *reinterpret_cast<const unsigned short*>(&v);
}
template <typename T, int V>
struct Pack {
  static constexpr int BYTES = (int)sizeof(T) * V;
  using W = std::conditional_t<BYTES % 4 == 0, unsigned, unsigned short>;
  static constexpr int NW = BYTES / (int)sizeof(W), PER = (int)(sizeof(W) / sizeof(T));
  alignas(BYTES < 16 ? BYTES : 16) W w[NW];

  __device__ __forceinline__ float get(int i) const {
    if constexpr (std::is_same_v<T, float>) {
      return __uint_as_float(w[i]);
    } else {
      const unsigned v = w[i / PER] >> (16 * (i % PER));
      if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        // a bfloat16 is the upper half of a float
        return __uint_as_float(PER == 2 && i % 2 ? w[i / PER] & 0xffff0000u : v << 16);
      } else {
        const unsigned short h = (unsigned short)v;
        return __half2float(*reinterpret_cast<const __half*>(&h));
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = 0;
  }
  // the i-th element, of a pack that is zero there
  __device__ __forceinline__ void put(int i, T v) { w[i / PER] |= (W)(bits_of(v) << (16 * (i % PER))); }
};

// V consecutive elements at p, of which `n` exist (the others read as 0 and are not
// written).  `vec`: p is a multiple of the pack's size, up to 16 bytes.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> ld_pack(const T* p, int n, bool vec) {
  Pack<T, V> r;
  using P = Pack<T, V>;
  if (vec && n >= V) {
    if (!touch(p, P::BYTES, P::BYTES < 16 ? P::BYTES : 16, false)) {
      r.zero();
      return r;
    }
    if constexpr (P::BYTES >= 16) {
#pragma unroll
      for (int i = 0; i < P::BYTES / 16; ++i)
        *reinterpret_cast<uint4*>(r.w + 4 * i) = reinterpret_cast<const uint4*>(p)[i];
    } else if constexpr (P::BYTES == 8) {
      *reinterpret_cast<uint2*>(r.w) = *reinterpret_cast<const uint2*>(p);
    } else {
      r.w[0] = *reinterpret_cast<const typename P::W*>(p);
    }
  } else {
    r.zero();
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) r.put(i, rd(p + i));
  }
  return r;
}
// The same where all of them exist and the address is aligned.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> ld_whole(const T* p) {
  return ld_pack<T, V>(p, V, true);
}
template <typename T, int V>
__device__ __forceinline__ void st_pack(T* p, int n, bool vec, const Pack<T, V>& r) {
  using P = Pack<T, V>;
  if (vec && n >= V) {
    if (!touch(p, P::BYTES, P::BYTES < 16 ? P::BYTES : 16, true)) return;
    if constexpr (P::BYTES >= 16) {
#pragma unroll
      for (int i = 0; i < P::BYTES / 16; ++i)
        reinterpret_cast<uint4*>(p)[i] = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
    } else if constexpr (P::BYTES == 8) {
      *reinterpret_cast<uint2*>(p) = make_uint2(r.w[0], r.w[1]);
    } else {
      *reinterpret_cast<typename P::W*>(p) = r.w[0];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i >= n) continue;
      if constexpr (sizeof(T) == 4)
        wr(reinterpret_cast<unsigned*>(p) + i, r.w[i]);
      else
        wr(reinterpret_cast<unsigned short*>(p) + i, (unsigned short)(r.w[i / P::PER] >> (16 * (i % P::PER))));
    }
  }
}
template <typename T, int V>
__device__ __forceinline__ void ld_f(const T* p, int n, bool vec, float (&v)[V]) {
  const Pack<T, V> r = ld_pack<T, V>(p, n, vec);
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = r.get(i);
}
// Two values rounded into one word.
template <typename T>
__device__ __forceinline__ unsigned two_of(float lo, float hi) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&r);
  } else {
    const __half2 r = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const unsigned*>(&r);
  }
}
template <typename T, int V>
__device__ __forceinline__ void st_f(T* p, int n, bool vec, const float (&v)[V]) {
  Pack<T, V> r;
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.w[i] = two_of<T>(v[2 * i], v[2 * i + 1]);
  } else {
    r.zero();
#pragma unroll
    for (int i = 0; i < V; ++i) r.put(i, from_f<T>(v[i]));
  }
  st_pack<T, V>(p, n, vec, r);
}

// A pack of an even number of elements as pairs.
template <typename T, int V>
__device__ __forceinline__ void to_pairs(const Pack<T, V>& r, float2 (&v)[V / 2]) {
#pragma unroll
  for (int i = 0; i < V / 2; ++i) v[i] = make_float2(r.get(2 * i), r.get(2 * i + 1));
}
template <typename T, int V>
__device__ __forceinline__ void st_pairs(T* p, int n, bool vec, const float2 (&v)[V / 2]) {
  float f[V];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    f[2 * i] = v[i].x;
    f[2 * i + 1] = v[i].y;
  }
  st_f<T, V>(p, n, vec, f);
}
template <typename T, int V>
__device__ __forceinline__ void st_whole(T* p, const float (&v)[V]) {
  st_f<T, V>(p, V, true, v);
}

// ---- packs on their way from global to shared memory -----------------------------------------
// A pack is copied asynchronously into a slot of the thread's own, which the thread alone reads
// back after fetched(): the next tile's data then waits in no registers.  Packs of less than 4
// bytes, and those that may not be read whole, go through registers.
template <typename T, int V>
__device__ __forceinline__ void fetch_whole(Pack<T, V>* slot, const T* src) {
  constexpr int BYTES = Pack<T, V>::BYTES;
  if (!touch(src, BYTES, BYTES < 16 ? BYTES : 16, false)) {
    slot->zero();
    return;
  }
  if constexpr (BYTES >= 4) {
#pragma unroll
    for (int i = 0; i < BYTES; i += 16)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(s4dev::smem_u32(slot) + i),
                   "l"(reinterpret_cast<const char*>(src) + i), "n"(BYTES < 16 ? BYTES : 16)
                   : "memory");
  } else
    *slot = ld_whole<T, V>(src);
}
// All but the thread's last N commits of copies are done (fetched(): all copies).
template <int N>
__device__ __forceinline__ void fetched_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void fetch_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// ---- packed pairs -----------------------------------------------------------------------
__device__ __forceinline__ unsigned long long u64(float2 v) { return *reinterpret_cast<unsigned long long*>(&v); }
__device__ __forceinline__ float2 f2(unsigned long long v) { return *reinterpret_cast<float2*>(&v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(u64(a)), "l"(u64(b)));
  return f2(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(u64(a)), "l"(u64(b)));
  return f2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(u64(a)), "l"(u64(b)), "l"(u64(c)));
  return f2(r);
}

// 2^v (relative error 2^-22, 0 for results below the normal range)
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float2 ex2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
constexpr float kLog2e = 1.44269504088896340736f;
// v sigmoid(v) and its derivative.  sigmoid = 1 / (1 + 2^(-v log2 e)) to about 2^-22, more for
// large negative v by |v| 2^-24 (the exponent's rounding); it tends to 0 and 1 without
// overflow trouble (2^.. = inf gives 0).
__device__ __forceinline__ float sigmoid(float v) { return s4dev::rcp_approx(1.f + ex2(v * -kLog2e)); }
__device__ __forceinline__ float2 sigmoid(float2 v) {
  const float2 e = add2(ex2(mul2(v, make_float2(-kLog2e, -kLog2e))), make_float2(1.f, 1.f));
  return make_float2(s4dev::rcp_approx(e.x), s4dev::rcp_approx(e.y));
}
__device__ __forceinline__ float silu(float v) { return v * sigmoid(v); }
__device__ __forceinline__ float2 silu(float2 v) { return mul2(v, sigmoid(v)); }
// silu' = s + silu (1 - s)
__device__ __forceinline__ float2 silu_grad(float2 v) {
  const float2 s = sigmoid(v), q = mul2(v, s);
  return fma2(q, fma2(s, make_float2(-1.f, -1.f), make_float2(1.f, 1.f)), s);
}

// The status block is optional in these calls (a null one records nothing).
__device__ __forceinline__ void record_gen(St st) {
  if (st.w) s4dev::st_record_gen(st);
}

// The state slot of sequence b (-1: none) and its real length.  A value out of range is
// recorded in the status and read as no slot and length 0.
struct Seq {
  long long slot;
  int len;
};
__device__ __forceinline__ Seq seq_of(const int* lengths, const int* index, int b, int L, int slots, St st) {
  Seq q;
  q.slot = index ? rd(index + b) : b;
  q.len = lengths ? rd(lengths + b) : L;
  const bool bad = q.len < 0 || q.len > L || (index && slots > 0 && q.slot >= slots);
  if (bad && st.w && threadIdx.x == 0) s4dev::st_flag(st, s4impl::ST_BAD_INDEX);
  if (bad || q.slot < 0) {
    q.slot = -1;
    q.len = 0;
  }
  return q;
}

// Sums over the lanes of a warp, in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// part[row][col], rows `pitch` floats apart, summed over the rows, columns in chunks of 32 per
// CTA, 8 row groups of one warp each; put(col, sum).
template <typename Put>
__device__ __forceinline__ void column_sums(const float* part, int rows, long long cols, long long pitch, Put put) {
  __shared__ float s[8][33];
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const long long c = (long long)blockIdx.x * 32 + lane;
  float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
  if (c < cols) {
    int r = wid;
    for (; r + 24 < rows; r += 32) {
      a0 += rd(part + r * pitch + c);
      a1 += rd(part + (r + 8) * pitch + c);
      a2 += rd(part + (r + 16) * pitch + c);
      a3 += rd(part + (r + 24) * pitch + c);
    }
    for (; r < rows; r += 8) a0 += rd(part + r * pitch + c);
  }
  s[wid][lane] = (a0 + a1) + (a2 + a3);
  __syncthreads();
  if (wid == 0 && c < cols) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += s[i][lane];
    put(c, t);
  }
}

// ---- host side ----------------------------------------------------------------------
// The current device (0 .. 63).
inline int device() {
  int dev = 0;
  return cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < 64 ? dev : 0;
}
// Lets a kernel have `bytes` of shared memory, once per device.
template <auto Kernel>
void allow_shared(int bytes) {
  static std::atomic<unsigned long long> done{0};
  const unsigned long long bit = 1ull << device();
  if (bytes <= 48 * 1024 || (done.load(std::memory_order_relaxed) & bit)) return;
  if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess)
    done.fetch_or(bit, std::memory_order_relaxed);
}
// Whether an array's accesses of `bytes` bytes are aligned: its address and its strides
// (in elements of `e` bytes).
inline bool vec_ok(const void* p, int e, int bytes, long long s0 = 0, long long s1 = 0) {
  return p == nullptr || ((uintptr_t)p % bytes == 0 && s0 * e % bytes == 0 && s1 * e % bytes == 0);
}

}  // namespace s4blk
