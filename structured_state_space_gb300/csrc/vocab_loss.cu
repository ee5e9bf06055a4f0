// Softmax cross entropy of hidden states against a vocabulary's weights, forward and backward, without
// keeping the logits x = w h:
//
//   lse = log sum_v e^{x_v},  loss = lse - x_target
//   g_v = dloss (e^{x_v - lse} - [v = target]),  dh = sum_v g_v w_v,  dw_v = sum_rows g_v h
//
// Forward: the tiles of the product h w^T are reduced where they are formed, each row of a tile to its maximum
// and its sum of exponentials, which a second kernel joins: 2 rows V H operations.  Backward: a piece of
// the vocabulary at a time, the logits are formed again and leave as g in 16-bit terms, which two more
// products take up: 6 rows V H operations.  The bound is the tensor cores.
//
// Measured in bfloat16: 1001 rows of 1024 channels and 32000 words 57 us forward (1.15 PFLOP/s), 8192 rows of 2048 and 50257 words
// 4.79 ms for losses and gradients (1.41 PFLOP/s; the forward product alone 1.77, of 1.71 that a library's
// sustains and 1.89 that it reaches in a burst); in float16 9.5 ms (g, h and w in two terms, three products each for dh and dw), in
// fp32 27 (six products each).  In fp32 with few channels the bound is g, three terms of it written once and read twice: 8192 rows
// of 64 and 32000 words 2.3 ms.
#include "s4_block.cuh"
#include "s4_sequence.h"
#include "tile_gemm.cuh"

namespace {
using namespace s4blk;
using namespace s4mma;

constexpr int kBN = 256;

// The target of a row: -1 where it does not count.
__device__ __forceinline__ long long target_of(const void* targets, int wide, long long row, int V, St st) {
  const long long t = wide ? rd(static_cast<const long long*>(targets) + row) : rd(static_cast<const int*>(targets) + row);
  if (t >= V) {
    s4dev::st_flag(st, s4impl::ST_BAD_INDEX);
    return -1;
  }
  return t < 0 ? -1 : t;
}

// Rows without a target whose hidden states are not finite, a bit each: their gradients of logits are zeros, and what they
// hold (padding may be NaN) is not to reach dw.
struct Padding {
  const unsigned long long* bits;  // [rows / 64, rounded up]
  __device__ __forceinline__ unsigned long long out(int chunk) const { return rd(bits + chunk); }
  __device__ __forceinline__ bool any(int from, int to) const {
    bool some = false;
    for (int c = from + (int)(threadIdx.x & 31); c < to; c += 32) some |= rd(bits + c) != 0;
    return __any_sync(0xffffffffu, some);
  }
};
size_t padding_bytes(long long rows) { return s4impl::section((size_t)(rows + 127) / 128 * 16); }

// ---- what becomes of a tile ---------------------------------------------------------------------------
// The maximum and the sum of exponentials (from it) of a row's logits in the tile, and the target's logit.
struct ToSums {
  float2* part;         // [tiles_n][rows]
  float* at_target;     // [rows]
  const void* targets;
  int wide, V;
  long long rows;
  St st;
  __device__ __forceinline__ void operator()(long long row, int n, int, uint32_t tmem) const {
    const bool live = row < rows;
    const long long t = live ? target_of(targets, wide, row, V, st) : -1;
    const int base = n * kBN, have = V - base < kBN ? V - base : kBN, want = t >= base && t < base + have ? (int)(t - base) : -1;
    float most = -INFINITY, sum = 0.f, hit = 0.f;
    uint32_t r[32];
#pragma unroll 1
    for (int c = 0; c < kBN; c += 32) {
      tmem_ld32(tmem + c, r);
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float x = __uint_as_float(r[i]);
        if (c + i < have) most = fmaxf(most, x);
        if (c + i == want) hit = x;
      }
    }
    const float off = most == -INFINITY ? 0.f : most * -kLog2e;
#pragma unroll 1
    for (int c = 0; c < have; c += 32) {
      tmem_ld32(tmem + c, r);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (c + i < have) sum += ex2(fmaf(__uint_as_float(r[i]), kLog2e, off));
    }
    if (!live) return;
    wr(part + n * rows + row, make_float2(most, sum));
    if (want >= 0) wr(at_target + row, hit);
  }
};

// The logits' gradients, in NP terms: g [NP][rows][pitch].
template <int NP>
struct ToGrads {
  __nv_bfloat16* g;
  unsigned* padding;    // see Padding, a word for the rows of a warp
  const float *lse, *dloss;
  const void* targets;
  int wide, V, first;   // the piece's first word
  long long rows, pitch;
  St st;
  __device__ __forceinline__ void operator()(long long row, int n, int, uint32_t tmem) const {
    const bool live = row < rows;
    const long long t = live ? target_of(targets, wide, row, V, st) : -1;
    const int base = first + n * kBN, have = V - base < kBN ? V - base : kBN;
    const int want = t >= base && t < base + kBN ? (int)(t - base) : -1;
    const float by = t >= 0 ? rd(dloss + row) : 0.f, off = live ? rd(lse + row) * -kLog2e : 0.f;
    if (n == 0) {
      // a row that is not finite has no finite logit, so no finite lse
      const unsigned bits = __ballot_sync(0xffffffffu, live && t < 0 && !(fabsf(off) < INFINITY));
      if ((threadIdx.x & 31) == 0) wr(padding + row / 32, bits);
    }
    __nv_bfloat16* to = g + row * pitch + n * kBN;
    uint32_t r[32];
#pragma unroll 1
    for (int c = 0; c < kBN; c += 32) {
      tmem_ld32(tmem + c, r);
      if (!live) continue;
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float e = ex2(fmaf(__uint_as_float(r[i + j]), kLog2e, off));
          v[j] = t >= 0 && c + i + j < have ? by * (c + i + j == want ? e - 1.f : e) : 0.f;
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          Pack<__nv_bfloat16, 8> w;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            w.w[j] = two_of<__nv_bfloat16>(v[2 * j], v[2 * j + 1]);
            v[2 * j] -= __uint_as_float(w.w[j] << 16);
            v[2 * j + 1] -= __uint_as_float(w.w[j] & 0xffff0000u);
          }
          st_pack<__nv_bfloat16, 8>(to + p * rows * pitch + c + i, 8, true, w);
        }
      }
    }
  }
};

// The values themselves, [splits][M][N] of T, or added to what is there (fp32).
template <typename T, bool ADD, int BN>
struct ToMatrix {
  T* out;
  int M, N;
  bool vec;
  __device__ __forceinline__ void operator()(long long row, int n, int split, uint32_t tmem) const {
    T* to = out + ((long long)split * M + row) * N + n * BN;
    const int have = N - n * BN;
    uint32_t r[32];
#pragma unroll 1
    for (int c = 0; c < BN && c < have; c += 32) {
      tmem_ld32(tmem + c, r);
      if (row >= M) continue;
#pragma unroll
      for (int i = 0; i < 32; i += 8) {
        if (c + i >= have) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(r[i + j]);
        if constexpr (ADD) {
          float old[8];
          ld_f<T, 8>(to + c + i, have - c - i, vec, old);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] += old[j];
        }
        st_f<T, 8>(to + c + i, have - c - i, vec, v);
      }
    }
  }
};

// ---- small kernels -------------------------------------------------------------------------------------
// A row's tiles joined, a warp per row.
__global__ void __launch_bounds__(256) join_kernel(const float2* part, const float* at_target, s4_vocab_loss_args a, int tiles,
                                                   St st) {
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= a.rows) return;
  float most = -INFINITY, sum = 0.f;
  bool nan = false;  // (a maximum leaves NaN out; the sums keep it)
  for (int i = lane; i < tiles; i += 32) {
    const float2 v = rd(part + i * a.rows + row);
    nan |= v.y != v.y;
    const float m = fmaxf(most, v.x);
    if (m != -INFINITY) sum = sum * ex2((most - m) * kLog2e) + v.y * ex2((v.x - m) * kLog2e);
    most = m;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, most, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
    const float m = fmaxf(most, m2);
    if (m != -INFINITY) sum = sum * ex2((most - m) * kLog2e) + s2 * ex2((m2 - m) * kLog2e);
    most = m;
  }
  nan = __any_sync(0xffffffffu, nan);
  if (lane != 0) return;
  const float lse = nan ? NAN : most == -INFINITY ? -INFINITY : most + logf(sum);
  const long long t = target_of(a.targets, a.wide_targets, row, a.V, st);
  wr(a.lse + row, lse);
  wr(a.loss + row, t >= 0 ? lse - rd(at_target + row) : 0.f);
}

// Rows of T as NP bfloat16 terms [NP][rows][pitch], zeros beyond H.  (NP = 1 of float16: as they are.)
template <typename T, int NP>
__global__ void __launch_bounds__(256) terms_kernel(const T* p, long long row, long long rows, int H, int pitch,
                                                    __nv_bfloat16* out, bool vec) {
  const long long packs = pitch / 8, n = rows * packs;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const long long r = i / packs;
    const int c = (int)(i - r * packs) * 8, have = H - c < 8 ? H - c : 8;
    const Pack<T, 8> v = ld_pack<T, 8>(p + r * row + c, have, vec);
    __nv_bfloat16* to = out + r * pitch + c;
    if constexpr (NP == 1) {
      Pack<__nv_bfloat16, 8> w;
#pragma unroll
      for (int j = 0; j < 4; ++j) w.w[j] = v.w[j];
      st_pack<__nv_bfloat16, 8>(to, 8, true, w);
    } else {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = v.get(j);
#pragma unroll
      for (int t = 0; t < NP; ++t) {
        Pack<__nv_bfloat16, 8> w;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w.w[j] = two_of<__nv_bfloat16>(f[2 * j], f[2 * j + 1]);
          f[2 * j] -= __uint_as_float(w.w[j] << 16);
          f[2 * j + 1] -= __uint_as_float(w.w[j] & 0xffff0000u);
        }
        st_pack<__nv_bfloat16, 8>(to + t * rows * pitch, 8, true, w);
      }
    }
  }
}

// Partial results summed in their order.
template <typename T>
__global__ void __launch_bounds__(256) splits_kernel(const float* part, int splits, long long n, T* out, bool vec) {
  for (long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 8; i < n; i += (long long)gridDim.x * 2048) {
    const int have = n - i < 8 ? (int)(n - i) : 8;
    float v[8];
    ld_f<float, 8>(part + i, have, true, v);
    for (int s = 1; s < splits; ++s) {
      float u[8];
      ld_f<float, 8>(part + s * n + i, have, n % 4 == 0, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += u[j];
    }
    st_f<T, 8>(out + i, have, vec, v);
  }
}

// ---- host side -----------------------------------------------------------------------------------------
int chunks_of(long long k) { return (int)((k + kBK - 1) / kBK); }
unsigned blocks_for(long long n) {
  const long long most = 16ll * s4impl::num_sms(), need = (n + 255) / 256;
  return (unsigned)(need < most ? need : most);
}

// A 16-bit operand [planes][rows][H] that tensor maps can have.
struct Operand {
  const void* p;
  long long row, plane, rows;
  int H, planes;
  bool bf16;
};
// Whether rows can go by TMA as they lie.
bool maps_take(const void* p, long long row, long long rows, int H, int e) {
  return e == 2 && (uintptr_t)p % 16 == 0 && (rows == 1 || (row >= H && row % 8 == 0 && row < (1ll << 36)));
}
int pitch_of(int H) { return (H + 7) / 8 * 8; }
size_t terms_bytes(long long rows, int H, int planes) { return s4impl::section((size_t)planes * rows * pitch_of(H) * 2); }

// What the products take of rows of T: themselves, or a copy in `planes` terms at `at` (1: of the same type).
template <typename T>
cudaError_t to_terms(const void* p, long long row, long long rows, int H, int planes, char* at, Operand* o, cudaStream_t s) {
  const int pitch = pitch_of(H);
  const bool vec = vec_ok(p, sizeof(T), 16, row);
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(at);
  *o = {at, pitch, (long long)pitch * rows, rows, H, planes, planes > 1 || std::is_same_v<T, __nv_bfloat16>};
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.add(p, sizeof(T), true, false, H, rows, row);
  x.scratch(at, 2, planes * rows * pitch);
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  const unsigned grid = blocks_for(rows * (pitch / 8));
  const T* in = static_cast<const T*>(p);
  s4impl::TimedLaunch tl("vocab_loss", s);
  if constexpr (sizeof(T) == 4) {
    terms_kernel<T, 3><<<grid, 256, 0, s>>>(in, row, rows, H, pitch, out, vec);
  } else {
    if (planes == 1)
      terms_kernel<T, 1><<<grid, 256, 0, s>>>(in, row, rows, H, pitch, out, vec);
    else
      terms_kernel<T, 2><<<grid, 256, 0, s>>>(in, row, rows, H, pitch, out, vec);
  }
  return cudaGetLastError();
}

// The plane pairs of a product of operands in `n` terms each: those whose sizes are above what the last term leaves
// out, the smallest first: the tensor cores cut what an addition shifts out of the accumulator, always
// towards zero, and while the small pairs are summed it is small.
void pairs_of(int n, Product* p) {
  p->pairs = 0;
  p->planes_a = p->planes_b = 0;
  for (int sum = n - 1; sum >= 0; --sum)
    for (int i = 0; i <= sum; ++i, ++p->pairs) {
      p->planes_a |= (uint32_t)i << (4 * p->pairs);
      p->planes_b |= (uint32_t)(sum - i) << (4 * p->pairs);
    }
}

// Sums in an accumulator drift, as the tensor cores cut off what an addition shifts out: about 1e-8 per addition of 16 k
// (measured).  In fp32 an accumulator takes up 1024 k and is then added, rounded, to a second one (off by 3e-7 to 6e-7; their
// six products hide the additions).  Logits of 16-bit inputs, whose lse is fp32 too, are summed in parts of 8192; gradients
// of float16 and bfloat16, off by up to 2^-11 and 2^-8 themselves, in products of 65536 and 262144 k (4e-5 and 2e-4).
constexpr int kPart = 16;  // chunks
int logits_part(int dtype) { return dtype == S4_F32 ? kPart : 128; }
int most_chunks(int dtype) { return dtype == S4_F32 ? 1 << 30 : dtype == S4_F16 ? 1024 : 4096; }

// result [M][N] = sum over k of A and B, in 64 k from chunk `first` on: A [M][k] or, A_MN, [k][M]; B likewise.
template <bool A_MN, bool B_MN, int BN = kBN, bool SUMMED = false, typename Epilogue, typename Counts = AllCount>
cudaError_t multiply(const Operand& a, const Operand& b, long long M, long long N, int first, int chunks, int splits,
                     const Epilogue& ep, St st, cudaStream_t s, const Counts& counts = {}, int part = 0) {
  constexpr auto kernel = product_kernel<BN, A_MN, B_MN, SUMMED, Epilogue, Counts>;
  CUtensorMap ma, mb;
  if (!make_map(&ma, a.p, a.bf16, a.H, a.rows, a.planes, a.row, a.plane, A_MN ? kBK : 128) ||
      !make_map(&mb, b.p, b.bf16, b.H, b.rows, b.planes, b.row, b.plane, B_MN ? kBK : BN))
    return cudaErrorInvalidValue;
  Product p{};
  p.M = (int)M, p.N = (int)N;
  p.tiles_m = (int)((M + 127) / 128), p.tiles_n = (int)((N + BN - 1) / BN);
  p.first = first, p.chunks = chunks;
  p.splits = splits, p.part = part;
  pairs_of(a.planes, &p);
  p.what = instruction(a.bf16, A_MN, B_MN, 128, BN);
  p.limit = s4impl::wait_limit();
  const long long tiles = (long long)p.tiles_m * p.tiles_n * splits;
  allow_shared<kernel>(Shape<BN>::BYTES);
  s4impl::TimedLaunch tl("vocab_loss", s);
  const unsigned grid = (unsigned)(tiles < s4impl::num_sms() ? tiles : s4impl::num_sms());
  kernel<<<grid, 256, Shape<BN>::BYTES, s>>>(ma, mb, p, ep, counts, st);
  return cudaGetLastError();
}

// The logits h w^T into `ep`.
template <typename Epilogue>
cudaError_t logits(const Operand& h, const Operand& w, int dtype, const Epilogue& ep, St st, cudaStream_t s) {
  const int chunks = chunks_of(h.H), part = logits_part(dtype);
  if (chunks > part) return multiply<false, false, kBN, true>(h, w, h.rows, w.rows, 0, chunks, 1, ep, st, s, AllCount{}, part);
  return multiply<false, false>(h, w, h.rows, w.rows, 0, chunks, 1, ep, st, s);
}

int terms_of(int dtype) { return dtype == S4_F32 ? 3 : dtype == S4_F16 ? 2 : 1; }

// Terms of the forward product: 16-bit types go as they are.
int logits_terms(int dtype) { return dtype == S4_F32 ? 3 : 1; }
// Bytes of the copies of h and w in n terms that a product needs.
template <typename Args>
size_t copies(const Args& a, int n) {
  const int e = s4impl::dtype_bytes(a.dtype);
  return (n == 1 && maps_take(a.h, a.h_row, a.rows, a.H, e) ? 0 : terms_bytes(a.rows, a.H, n)) +
         (n == 1 && maps_take(a.w, a.w_row, a.V, a.H, e) ? 0 : terms_bytes(a.V, a.H, n));
}
template <typename T>
cudaError_t operand(const void* p, long long row, long long rows, int H, int planes, char** at, Operand* o, cudaStream_t s) {
  if (maps_take(p, row, rows, H, sizeof(T)) && planes == 1) {
    const long long pitch = rows == 1 ? pitch_of(H) : row;
    *o = {p, pitch, pitch, rows, H, 1, std::is_same_v<T, __nv_bfloat16>};
    return cudaSuccess;
  }
  char* to = *at;
  *at += terms_bytes(rows, H, planes);
  return to_terms<T>(p, row, rows, H, planes, to, o, s);
}

template <typename T>
cudaError_t fwd_t(const s4_vocab_loss_args& a, St st, cudaStream_t s) {
  char* at = static_cast<char*>(a.ws) + s4impl::kStatusBytes;
  const int tiles_n = (a.V + kBN - 1) / kBN, n = logits_terms(a.dtype);
  float2* part = reinterpret_cast<float2*>(at);
  at += s4impl::section(sizeof(float2) * tiles_n * a.rows);
  float* hit = reinterpret_cast<float*>(at);
  at += s4impl::section(sizeof(float) * a.rows);
  Operand h, w;
  cudaError_t err = operand<T>(a.h, a.h_row, a.rows, a.H, n, &at, &h, s);
  if (err != cudaSuccess) return err;
  err = operand<T>(a.w, a.w_row, a.V, a.H, n, &at, &w, s);
  if (err != cudaSuccess) return err;
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.in(a.targets, a.wide_targets ? 8 : 4, a.rows);
  x.scratch(part, 8, tiles_n * a.rows);
  x.scratch(hit, 4, a.rows);
  x.out(a.loss, 4, a.rows);
  x.out(a.lse, 4, a.rows);
  if (const cudaError_t e = set_extents(x, s); e != cudaSuccess) return e;
#endif
  const ToSums ep{part, hit, a.targets, a.wide_targets, a.V, a.rows, st};
  err = logits(h, w, a.dtype, ep, st, s);
  if (err != cudaSuccess) return err;
  s4impl::TimedLaunch tl("vocab_loss", s);
  join_kernel<<<(unsigned)((a.rows + 7) / 8), 256, 0, s>>>(part, hit, a, tiles_n, st);
  return cudaGetLastError();
}

// Words per piece: gradients of the logits of up to 512 MB, in whole tiles (8192 rows of 2048 channels, 50257 words: 4.78 ms
// with the forward pass; pieces of 256 MB 4.86, of 128 MB 4.99: more, and fuller, rounds of tiles in a piece).
constexpr size_t kPieceBytes = 512ull << 20;
long long piece_words(long long rows, int V, int planes) {
  long long n = (long long)(kPieceBytes / (2ull * planes * rows)) / kBN * kBN;
  if (n < kBN) n = kBN;
  const long long all = (V + kBN - 1ll) / kBN * kBN, pieces = (all + n - 1) / n;
  return (all / kBN + pieces - 1) / pieces * kBN;  // of nearly equal sizes
}
// Columns of the tiles of a product [M][N] (gradients of 8192 rows of 64 channels and 32000 words in fp32: with 64 columns 2.16
// ms, with 256 2.35).
int columns(long long N) { return N <= 64 ? 64 : N <= 128 ? 128 : 256; }
// Shares of the sum over k of a product [M][N]: where its tiles are fewer than the SMs.
int shares(long long M, long long N, long long k) {
  const long long tiles = (M + 127) / 128 * ((N + columns(N) - 1) / columns(N)), chunks = chunks_of(k);
  long long n = s4impl::num_sms() / tiles;
  if (n > chunks / 8) n = chunks / 8;
  return n < 1 ? 1 : (int)n;
}
// out (+)= A B: in one product where it can go straight out (`part` is then not used, and nothing may be added later),
// else as `splits` partial results in part [splits][M][N].
template <typename T, bool A_MN, int BN, typename Counts>
cudaError_t sum_products_n(const Operand& a, const Operand& b, long long M, long long N, long long K, int splits, bool add,
                           bool direct, T* out, float* part, St st, cudaStream_t s, const Counts& counts) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int code = F32 ? S4_F32 : std::is_same_v<T, __half> ? S4_F16 : S4_BF16;
  const int chunks = chunks_of(K);
  const long long most = (long long)most_chunks(code) * splits;
  if (direct && chunks <= most) {
    const ToMatrix<T, false, BN> ep{out, (int)M, (int)N, N % 8 == 0 && vec_ok(out, sizeof(T), 16)};
    return multiply<A_MN, true, BN, F32>(a, b, M, N, 0, chunks, 1, ep, st, s, counts, kPart);
  }
  const bool vec = N % 4 == 0 && vec_ok(part, 4, 16);
  for (int first = 0; first < chunks; first += (int)most, add = true) {
    const int n = chunks - first < most ? chunks - first : (int)most;
    const ToMatrix<float, true, BN> more{part, (int)M, (int)N, vec};
    const ToMatrix<float, false, BN> begin{part, (int)M, (int)N, vec};
    const cudaError_t err = add ? multiply<A_MN, true, BN, F32>(a, b, M, N, first, n, splits, more, st, s, counts, kPart)
                                : multiply<A_MN, true, BN, F32>(a, b, M, N, first, n, splits, begin, st, s, counts, kPart);
    if (err != cudaSuccess) return err;
    if (n == chunks - first) break;
  }
  return cudaSuccess;
}
template <typename T, bool A_MN, typename Counts = AllCount>
cudaError_t sum_products(const Operand& a, const Operand& b, long long M, long long N, long long K, int splits, bool add,
                         bool direct, T* out, float* part, St st, cudaStream_t s, const Counts& counts = {}) {
  switch (columns(N)) {
    case 64: return sum_products_n<T, A_MN, 64>(a, b, M, N, K, splits, add, direct, out, part, st, s, counts);
    case 128: return sum_products_n<T, A_MN, 128>(a, b, M, N, K, splits, add, direct, out, part, st, s, counts);
    default: return sum_products_n<T, A_MN, 256>(a, b, M, N, K, splits, add, direct, out, part, st, s, counts);
  }
}
template <typename T>
cudaError_t add_up(const float* part, int splits, long long n, T* out, cudaStream_t s) {
  s4impl::TimedLaunch tl("vocab_loss", s);
  splits_kernel<T><<<blocks_for(n / 8 + 1), 256, 0, s>>>(part, splits, n, out, vec_ok(out, sizeof(T), 16));
  return cudaGetLastError();
}

// What a backward pass has beside the operands' copies.
struct Plan {
  long long words, pieces;
  int dh_splits, dw_splits;
  size_t g, dh, dw, padding;  // bytes
};
template <typename Args>
Plan plan_of(const Args& a) {
  Plan p;
  const int np = terms_of(a.dtype);
  p.words = piece_words(a.rows, a.V, np), p.pieces = (a.V + p.words - 1) / p.words;
  p.dh_splits = shares(a.rows, a.H, p.words), p.dw_splits = shares(p.words, a.H, a.rows);
  p.g = s4impl::section(2ull * np * a.rows * p.words);
  const int most = most_chunks(a.dtype);
  p.dh = p.pieces > 1 || p.dh_splits > 1 || chunks_of(p.words) > most ? s4impl::section(4ull * p.dh_splits * a.rows * a.H) : 0;
  p.dw = p.dw_splits > 1 || chunks_of(a.rows) > most ? s4impl::section(4ull * p.dw_splits * p.words * a.H) : 0;
  p.padding = padding_bytes(a.rows);
  return p;
}

template <typename T>
cudaError_t bwd_t(const s4_vocab_loss_bwd_args& a, St st, cudaStream_t s) {
  constexpr int NP = sizeof(T) == 4 ? 3 : std::is_same_v<T, __half> ? 2 : 1;
  const Plan p = plan_of(a);
  const long long words = p.words;
  char* at = static_cast<char*>(a.ws) + s4impl::kStatusBytes;
  __nv_bfloat16* g = reinterpret_cast<__nv_bfloat16*>(at);
  at += p.g;
  float* dh = reinterpret_cast<float*>(at);
  at += p.dh;
  float* dw = reinterpret_cast<float*>(at);
  at += p.dw;
  unsigned* padding = reinterpret_cast<unsigned*>(at);
  at += p.padding;
  Operand h, w, lh, lw;
  cudaError_t err = operand<T>(a.h, a.h_row, a.rows, a.H, NP, &at, &h, s);
  if (err != cudaSuccess) return err;
  err = operand<T>(a.w, a.w_row, a.V, a.H, NP, &at, &w, s);
  if (err != cudaSuccess) return err;
  lh = h, lw = w;
  if (std::is_same_v<T, __half>) {
    // the logits' product takes float16 as it is, as in the forward pass
    err = operand<T>(a.h, a.h_row, a.rows, a.H, 1, &at, &lh, s);
    if (err != cudaSuccess) return err;
    err = operand<T>(a.w, a.w_row, a.V, a.H, 1, &at, &lw, s);
    if (err != cudaSuccess) return err;
  }
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  x.in(a.targets, a.wide_targets ? 8 : 4, a.rows);
  x.in(a.lse, 4, a.rows);
  x.in(a.dloss, 4, a.rows);
  x.scratch(g, 2, NP * a.rows * words);
  if (p.dh) x.scratch(dh, 4, p.dh_splits * a.rows * a.H);
  if (p.dw) x.scratch(dw, 4, p.dw_splits * words * a.H);
  x.scratch(padding, 4, (a.rows + 127) / 128 * 4);
  x.out(a.dh, sizeof(T), a.rows * a.H);
  x.out(a.dw, sizeof(T), (long long)a.V * a.H);
  if (const cudaError_t e = set_extents(x, s); e != cudaSuccess) return e;
#endif
  const auto rows_from = [](const Operand& o, long long first, long long n) {
    Operand r = o;
    r.p = static_cast<const char*>(o.p) + first * o.row * 2;
    r.rows = n;
    return r;
  };
  const Padding counts{reinterpret_cast<const unsigned long long*>(padding)};
  for (long long first = 0; first < a.V; first += words) {
    const long long n = a.V - first < words ? a.V - first : words;
    const ToGrads<NP> grads{g, padding, a.lse, a.dloss, a.targets, a.wide_targets, a.V, (int)first, a.rows, words, st};
    err = logits(lh, rows_from(lw, first, n), a.dtype, grads, st, s);
    if (err != cudaSuccess) return err;
    const Operand gr{g, words, words * a.rows, a.rows, (int)n, NP, true};
    T* to_w = static_cast<T*>(a.dw) + first * a.H;
    err = sum_products<T, true>(gr, h, n, a.H, a.rows, p.dw_splits, false, !p.dw, to_w, dw, st, s, counts);
    if (err == cudaSuccess && p.dw) err = add_up<T>(dw, p.dw_splits, n * a.H, to_w, s);
    if (err != cudaSuccess) return err;
    err = sum_products<T, false>(gr, rows_from(w, first, n), a.rows, a.H, n, p.dh_splits, first > 0, !p.dh,
                                       static_cast<T*>(a.dh), dh, st, s);
    if (err != cudaSuccess) return err;
  }
  return p.dh ? add_up<T>(dh, p.dh_splits, a.rows * a.H, static_cast<T*>(a.dh), s) : cudaSuccess;
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_vocab_loss)
#endif

size_t vocab_loss_scratch(const s4_vocab_loss_args& a) {
  return section(sizeof(float2) * ((a.V + kBN - 1) / kBN) * a.rows) + section(sizeof(float) * a.rows) +
         copies(a, logits_terms(a.dtype));
}

cudaError_t launch_vocab_loss(const s4_vocab_loss_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return fwd_t<float>(a, st, s);
  return a.dtype == S4_BF16 ? fwd_t<__nv_bfloat16>(a, st, s) : fwd_t<__half>(a, st, s);
}

size_t vocab_loss_bwd_scratch(const s4_vocab_loss_bwd_args& a) {
  const Plan p = plan_of(a);
  size_t n = p.g + p.dh + p.dw + p.padding + copies(a, terms_of(a.dtype));
  if (a.dtype == S4_F16) n += copies(a, 1);
  return n;
}

cudaError_t launch_vocab_loss_bwd(const s4_vocab_loss_bwd_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float>(a, st, s);
  return a.dtype == S4_BF16 ? bwd_t<__nv_bfloat16>(a, st, s) : bwd_t<__half>(a, st, s);
}

}  // namespace s4impl
