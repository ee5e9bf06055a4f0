// Tiles of matrix products on the fifth-generation tensor cores: accumulators of 128 x BN in tensor
// memory, operands of 16 bits brought by TMA into shared memory with the 128-byte swizzle.
//
// An operand lies in memory either with the summed dimension k contiguous ("K-major": tiles of
// rows x 64 k) or with its other dimension contiguous ("MN-major": blocks of 64 columns x 64 k).
// Both may come as several terms (planes) whose sum is the operand: a product then runs over
// the list of plane pairs, all into one accumulator.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "s4_dev.cuh"

namespace s4mma {

constexpr int kBK = 64;  // elements of k per stage: one 128-byte row of the swizzle

// ---- descriptors -----------------------------------------------------------------------------------
// Instruction descriptor of kind::f16 with fp32 accumulators: types (0: float16, 1: bfloat16), majors, sizes.
__host__ __device__ constexpr uint32_t instruction(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}
// Shared-memory descriptor of a 128-byte swizzled tile: 1024 bytes from one group of 8 rows to the next;
// MN-major tiles have `lead` bytes between blocks of 64 columns.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)(addr >> 4 & 0x3fff) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// ---- instructions ----------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, int cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(s4dev::smem_u32(slot)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}
// Products and commits are issued by the one lane of a warp that has `one` set.  They are predicated, not under a branch:
// the warp stays together and its descriptors in uniform registers (under a branch an issue took about twice as long).
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t what, bool add, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(what), "r"((uint32_t)add), "r"(one)
      : "memory");
}
// Arrives at the barrier when all products issued so far are done.
__device__ __forceinline__ void mma_commit(unsigned long long* bar, uint32_t one) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(s4dev::smem_u32(bar)),
      "r"(one)
      : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 columns of the warp's 32 lanes: thread l has lane l's row.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
      "[%32];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
// Twice as much, on its way at once.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t at2, uint32_t (&r)[32], uint32_t (&q)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15]), "=r"(q[16]), "=r"(q[17]), "=r"(q[18]), "=r"(q[19]), "=r"(q[20]), "=r"(q[21]), "=r"(q[22]), "=r"(q[23]), "=r"(q[24]), "=r"(q[25]), "=r"(q[26]), "=r"(q[27]), "=r"(q[28]), "=r"(q[29]), "=r"(q[30]), "=r"(q[31])
      : "r"(at), "r"(at2)
      : "memory");
}
// 16 columns of two places, on their way at once, and 16 written.
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t at2, uint32_t (&r)[16], uint32_t (&q)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(q[0]), "=r"(q[1]), "=r"(q[2]),
        "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]),
        "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15])
      : "r"(at), "r"(at2)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y, int z, unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          s4dev::smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(s4dev::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void arrive(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(s4dev::smem_u32(bar)) : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// ---- the product -----------------------------------------------------------------------------------
struct Product {
  int M, N;                 // of the result
  int tiles_m, tiles_n;     // of 128 x BN
  int first, chunks;        // of 64 k: where they begin, how many
  int splits;               // the chunks are shared out among so many partial results
  int part;                 // chunks that an accumulator takes up before it is added to the sum (SUMMED)
  int pairs;                // plane pairs: nibble p of each list
  uint32_t planes_a, planes_b;
  uint32_t what;            // instruction descriptor
  int limit;                // polls of a wait before it gives up
};

template <int BN>
struct Shape {
  static constexpr int A = 128 * kBK * 2, B = BN * kBK * 2, STAGE = A + B;  // bytes
  static constexpr int STAGES = BN == 256 ? 4 : 6;
  static constexpr int BYTES = STAGES * STAGE + 1024;                       // dynamic shared memory, with its alignment
  static constexpr int COLS = 2 * BN;                                       // of tensor memory: two accumulators
};

// Which k of a product do not count, a bit for each of a chunk's, and whether there are any in chunks [from, to): none.
struct AllCount {
  __device__ __forceinline__ unsigned long long out(int) const { return 0; }
  __device__ __forceinline__ bool any(int, int) const { return false; }
};

// 256 threads: warp 0 brings the operands, warp 1 issues the products, warps 4 to 7 take the results
// from one accumulator while the other is filled.  Where some k do not count (with an MN-major B), A is zero there
// and B may hold anything, NaN too: warp 1 blanks B's rows of them in shared memory before it multiplies.  Every wait
// is bounded; where one gives up the CTA records a stall, waits for its copies and products in flight, frees
// its tensor memory and leaves.  SUMMED: an accumulator takes up a part of the chunks at a time, and the second one is the sum
// of the parts, added rounded (the tensor cores cut what an addition shifts out, so long sums in one drift).
template <int BN, bool A_MN, bool B_MN, bool SUMMED, typename Epilogue, typename Counts>
__global__ void __launch_bounds__(256, 1)
    product_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const Product p,
                   const Epilogue ep, const Counts counts, s4impl::St st) {
  using S = Shape<BN>;
  extern __shared__ char raw[];
  __shared__ unsigned long long full[S::STAGES], empty[S::STAGES], ready[2], taken[2], idle;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int failed;
  char* smem = raw + (-s4dev::smem_u32(raw) & 1023);  // (still a shared-memory address to the compiler)
  const int wid = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform)
  if (st.w) s4dev::st_record_gen(st);
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::STAGES; ++i) s4dev::mbar_init(&full[i], 1), s4dev::mbar_init(&empty[i], 1);
    for (int i = 0; i < 2; ++i) s4dev::mbar_init(&ready[i], 1), s4dev::mbar_init(&taken[i], 4);
    s4dev::mbar_init(&idle, 1);
    failed = 0;
    s4dev::fence_mbar_init();
  }
  if (wid == 1) tmem_alloc(&tmem_slot, S::COLS);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = S::COLS == 512 ? 0 : tmem_slot;  // (all of it begins at 0)
  const int tiles = p.tiles_m * p.tiles_n * p.splits;
  const auto wait = [&](unsigned long long* bar, unsigned parity) {
    for (int it = 0; it < p.limit; it += 256) {
      if (s4dev::mbar_wait(bar, parity, p.limit - it < 256 ? p.limit - it : 256)) return true;
      if (failed) return false;
    }
    failed = 1;
    return false;
  };
  const auto wait_warp = [&](unsigned long long* bar, unsigned parity) {
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };
  struct Tile {
    int m, n, from, to, split;
  };
  // m runs fastest: CTAs of one time share the tiles of B, and A's all fit the L2
  const auto tile_of = [&](int t) {
    Tile r;
    r.m = t % p.tiles_m;
    r.n = t / p.tiles_m % p.tiles_n;
    r.split = t / p.tiles_m / p.tiles_n;
    r.from = p.first + (int)((long long)p.chunks * r.split / p.splits);
    r.to = p.first + (int)((long long)p.chunks * (r.split + 1) / p.splits);
    return r;
  };

  const int part = SUMMED ? p.part : p.chunks;
  int issued = 0;  // rounds of copies
  if (wid == 0 && elected()) {
    int stage = 0;
    unsigned phase = 0;
    for (int t = blockIdx.x; t < tiles && !failed; t += gridDim.x) {
      const Tile at = tile_of(t);
      for (int from = at.from, i = 0; from < at.to && !failed; i = i + 1 == p.pairs ? 0 : i + 1, from += i == 0 ? part : 0) {
        const int za = p.planes_a >> (4 * i) & 15, zb = p.planes_b >> (4 * i) & 15, to = from + part < at.to ? from + part : at.to;
        for (int c = from; c < to; ++c) {
          if (!wait(&empty[stage], phase ^ 1)) break;
          char* a = smem + stage * S::STAGE;
          char* b = a + S::A;
          s4dev::mbar_expect_tx(&full[stage], S::STAGE);
          if (A_MN) {
#pragma unroll
            for (int x = 0; x < 2; ++x) tma_load(a + x * 8192, &map_a, at.m * 128 + 64 * x, c * kBK, za, &full[stage]);
          } else {
            tma_load(a, &map_a, c * kBK, at.m * 128, za, &full[stage]);
          }
          if (B_MN) {
#pragma unroll
            for (int x = 0; x < BN / 64; ++x) tma_load(b + x * 8192, &map_b, at.n * BN + 64 * x, c * kBK, zb, &full[stage]);
          } else {
            tma_load(b, &map_b, c * kBK, at.n * BN, zb, &full[stage]);
          }
          ++issued;
          if (++stage == S::STAGES) stage = 0, phase ^= 1;
        }
      }
    }
  } else if (wid == 1) {
    // the warp stays together, so that the descriptors are uniform; one lane issues
    const uint32_t one = elected();
    int stage = 0, buf = 0;
    unsigned phase = 0, buf_phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile at = tile_of(t);
      const bool blanks = counts.any(at.from, at.to);
      // (where there is nothing to sum up the results' warps are told so once, but not of parts)
      for (int from = at.from; ok && (from < at.to || (!SUMMED && from == at.from)); from += part) {
        const int n = (from + part < at.to ? from + part : at.to) - from;
        ok = wait_warp(&taken[buf], buf_phase ^ 1);
        fence_after();
        const uint32_t d = tmem + buf * BN;
        const int steps = ok ? p.pairs * n : 0;
        for (int i = 0; i < steps; ++i) {
          ok = wait_warp(&full[stage], phase);
          if (!ok) break;
          fence_after();
          const uint32_t a = s4dev::smem_u32(smem) + stage * S::STAGE, b = a + S::A;
          if (blanks) {
            // a row of k has 128 bytes in each block of 64 columns: 16 bytes a lane
            char* at_lane = smem + stage * S::STAGE + S::A + lane / 8 * 8192 + lane % 8 * 16;
            for (unsigned long long left = counts.out(from + i % n); left; left &= left - 1)
              if (lane < BN / 8) *reinterpret_cast<uint4*>(at_lane + (__ffsll(left) - 1) * 128) = make_uint4(0, 0, 0, 0);
            s4dev::fence_proxy_async();
            __syncwarp();
          }
          const uint64_t da = tile_desc(a, A_MN ? 8192 : 16), db = tile_desc(b, B_MN ? 8192 : 16);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            mma_f16(d, da + k * (A_MN ? 2048 >> 4 : 32 >> 4), db + k * (B_MN ? 2048 >> 4 : 32 >> 4), p.what, i + k > 0, one);
          mma_commit(&empty[stage], one);
          if (++stage == S::STAGES) stage = 0, phase ^= 1;
        }
        if (ok) mma_commit(&ready[buf], one);
        if (SUMMED || ++buf == 2) buf = 0, buf_phase ^= 1;
      }
    }
  } else if (wid >= 4) {
    int buf = 0;
    unsigned buf_phase = 0;
    const uint32_t lanes = tmem + ((uint32_t)(wid & 3) * 32 << 16);
    bool ok = true;
    for (int t = blockIdx.x; t < tiles && ok; t += gridDim.x) {
      const Tile at = tile_of(t);
      const int row = at.m * 128 + (wid & 3) * 32 + lane;
      if constexpr (SUMMED) {
        for (int from = at.from; from < at.to; from += part) {
          ok = wait_warp(&ready[0], buf_phase);
          if (!ok) break;
          buf_phase ^= 1;
          fence_after();
#pragma unroll 1
          for (int c = 0; c < BN; c += 16) {
            uint32_t r[16], q[16];
            tmem_ld16(lanes + c, lanes + BN + c, r, q);
            if (from > at.from) {
#pragma unroll
              for (int x = 0; x < 16; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) + __uint_as_float(q[x]));
            }
            tmem_st16(lanes + BN + c, r);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          fence_before();
          __syncwarp();
          if (lane == 0) arrive(&taken[0]);
        }
        if (ok && at.from < at.to) ep(row, at.n, at.split, lanes + BN);
      } else {
        ok = wait_warp(&ready[buf], buf_phase);
        if (!ok) break;
        fence_after();
        if (at.from < at.to)  // (a last piece may have fewer chunks than splits)
          ep(row, at.n, at.split, lanes + buf * BN);
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(&taken[buf]);
        if (++buf == 2) buf = 0, buf_phase ^= 1;
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (failed) {
    // the copies and products in flight: the last rounds of the stages
    if (threadIdx.x == 0 && st.w) s4dev::st_flag(st, s4dev::ST_STALL);
    for (int j = issued > S::STAGES ? issued - S::STAGES : 0; j < issued; ++j)
      s4dev::mbar_wait(&full[j % S::STAGES], (unsigned)(j / S::STAGES) & 1);
    if (wid == 1) {
      mma_commit(&idle, elected());
      s4dev::mbar_wait(&idle, 0);
    }
    fence_before();
    __syncthreads();
    fence_after();
  }
  if (wid == 1) tmem_free(tmem, S::COLS);
}

// ---- host side -------------------------------------------------------------------------------------
// The driver's cuTensorMapEncodeTiled (null where it has none), asked for once.
inline void* map_encoder() {
  static void* const f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r);
    return e == cudaSuccess && r == cudaDriverEntryPointSuccess ? p : nullptr;
  }();
  return f;
}

// A 16-bit array [planes][rows][width] as boxes of 64 x `box_rows`; false where a map cannot have it.
inline bool make_map(CUtensorMap* map, const void* p, bool bf16, long long width, long long rows, int planes, long long row,
                     long long plane, int box_rows) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const Encode encode = reinterpret_cast<Encode>(map_encoder());
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)planes};
  const cuuint64_t strides[2] = {(cuuint64_t)row * 2, (cuuint64_t)plane * 2};
  const cuuint32_t box[3] = {kBK, (cuuint32_t)box_rows, 1}, unit[3] = {1, 1, 1};
  return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims,
                strides, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace s4mma
