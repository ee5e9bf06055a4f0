// The walks of linear attention (linear_attention.cu) on the fifth-generation tensor cores, for bfloat16 and
// widths up to 128: chunks of 128 tokens, per chunk
//
//   S = A B^T,  P = S with the decays e^{g lag} (0 for later tokens), O = P C + e_i A M,  D = (f_j B)^T C,  M' = e^{g n} M + D
//
// with the accumulators S, O (two parts), D in tensor memory, P beside S as a left operand, and the state M in the
// registers of one warpgroup (thread r has row r), rounded into shared memory where A multiplies it.  The scaled
// keys f_j B enter the fp32 state as NK bfloat16 terms: 2 where the state only makes bfloat16 outputs, 3 where
// it is returned.
//
// Per chunk at widths 128: S, P C and A M 2^22 operations each, D 2^22 a term, which takes 1.7 to 2 us of an SM's share of
// the measured rate; the inputs and the output are 128 KB, 2.9 us of an SM's share of the memory's.  Measured on 4 x 4096
// tokens of 16 heads of 128: 219 us for the three walks of a backward pass, 3.4 us a chunk on 152 SMs at once; what is
// above the memory's share are 40 of 192 walks left for a second round, and three walks that read 12 arrays
// where one would read 7.  65536 tokens of 16 heads of 64 take 266 us, 2.8 us a chunk (64 KB, 1.4 us): there
// the warp that issues the products is the bound, 40 of them per chunk at 90 cycles or so (a right operand of 64
// columns does not feed the tensor cores), and a walk over segments reads keys and values twice.  Outputs spill 24 to 48
// bytes a thread at the 128 registers that four warpgroups start with (140 to 236 bytes loaded again).
#include "linear_attention.cuh"
#include "tile_gemm.cuh"

namespace {
using namespace s4blk;
using namespace s4mma;
using s4impl::In;
using s4impl::Walk;
using s4impl::Walks;

// Why so: accumulators of 128 lanes want 128 tokens; with 64 the products' tiles are half empty.  One warpgroup for P, O and
// the keys together took 11.9 thousand cycles a chunk, two 6.4, three 6.6 with keys and state side by side (and half
// the time where the state is returned); stores to global memory straight from the accumulators' lanes, 32
// rows an instruction, slowed the keys' shared-memory traffic to a third: outputs go through shared memory.
constexpr int kC = 128, kSlot = 32, kPasses = 3, kThreads = 512;

struct Maps {
  CUtensorMap a, b, c, out;  // (out: bfloat16 outputs whose strides a map can have)
};
struct Passes {
  Maps maps[kPasses];
  Walks walks;
  bool by_map[kPasses];  // whether whole chunks of outputs go by their map
  int limit;
};

template <int DK, int DV, int NK, bool STATE>
struct Room {
  static constexpr int TA = kC * DK * 2, TC = kC * DV * 2, TM = DK * DV * 2;  // bytes of a tile
  static constexpr int SA = STATE ? 0 : DK == 64 ? 2 : 1, SB = DK == 64 || STATE || (DV == 128 && NK == 2) ? 2 : 1;
  static constexpr int SC = DK == 128 && DV == 128 && !STATE ? 1 : 2;
  // scaled keys in slots of 32 tokens
  static constexpr int TK = kSlot * DK * 2, SK = DK == 128 && DV == 128 && !STATE ? 2 : 4;
  static constexpr int A = 0, B = A + SA * TA, C = B + SB * TA, K = C + SC * TC, M = K + SK * NK * TK;
  // outputs go through shared memory where it has room for them
  static constexpr bool STAGED = !STATE && M + TM + TC <= 224 * 1024;
  static constexpr int O = M + (STATE ? 0 : TM), BYTES = O + (STAGED ? TC : 0) + 1024;
  // columns of tensor memory
  static constexpr int S = 0, O1 = 128, O2 = O1 + DV, D = O2 + DV, COLS = 512;
};

__device__ __forceinline__ void mma_tmem_a(uint32_t d, uint32_t a, uint64_t b, uint32_t what, bool add, uint32_t one) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}" ::"r"(d),
      "r"(a), "l"(b), "r"(what), "r"((uint32_t)add), "r"(one)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int head, int t, int b,
                                            unsigned long long* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          s4dev::smem_u32(dst)),
      "l"(map), "r"(x), "r"(head), "r"(t), "r"(b), "r"(s4dev::smem_u32(bar))
      : "memory");
}

// 32 columns of a row, `have` of them there.
__device__ __forceinline__ void put_row(void* out, long long at, int have, bool f32, bool vec, const float2 (&f)[16]) {
  if (vec && have >= 32) {
    if (!f32) {
#pragma unroll
      for (int x = 0; x < 16; x += 4) {
        Pack<__nv_bfloat16, 8> v;
#pragma unroll
        for (int y = 0; y < 4; ++y) v.w[y] = two_of<__nv_bfloat16>(f[x + y].x, f[x + y].y);
        st_pack<__nv_bfloat16, 8>(static_cast<__nv_bfloat16*>(out) + at + 2 * x, 8, true, v);
      }
    } else {
#pragma unroll
      for (int x = 0; x < 16; x += 2) {
        const float v[4] = {f[x].x, f[x].y, f[x + 1].x, f[x + 1].y};
        st_whole<float, 4>(static_cast<float*>(out) + at + 2 * x, v);
      }
    }
    return;
  }
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    if (x >= have) return;
    const float v = x % 2 ? f[x / 2].y : f[x / 2].x;
    if (f32)
      wr(static_cast<float*>(out) + at + x, v);
    else
      wr(static_cast<__nv_bfloat16*>(out) + at + x, from_f<__nv_bfloat16>(v));
  }
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int head, int t, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(map),
               "r"(s4dev::smem_u32(src)), "r"(x), "r"(head), "r"(t), "r"(b)
               : "memory");
}
// Whether all of the first warpgroup's threads say so.
__device__ __forceinline__ bool all_of(bool v) {
  uint32_t r;
  asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %1, 0;\n barrier.cta.red.and.pred q, 1, 128, p;\n selp.b32 %0, 1, 0, q;\n}"
               : "=r"(r)
               : "r"((uint32_t)v)
               : "memory");
  return r != 0;
}
// An arrival that orders no earlier writes (stores to global memory, on which it would wait).
__device__ __forceinline__ void arrive_relaxed(unsigned long long* bar) {
  asm volatile("mbarrier.arrive.relaxed.cta.shared::cta.b64 _, [%0];" ::"r"(s4dev::smem_u32(bar)) : "memory");
}

// What all of a CTA's threads know of its walk.
struct Span {
  int begin, end, chunks;  // tokens in the order of memory
  bool last;               // the walk ends in this segment
};
__device__ __forceinline__ Span span_of(const Walk& w, int seg, int len) {
  const int live = (len + w.seg - 1) / w.seg, at = w.reverse ? live - 1 - seg : seg;
  Span p;
  p.begin = at * w.seg;
  p.end = p.begin + w.seg < len ? p.begin + w.seg : len;
  p.chunks = seg < live ? (p.end - p.begin + kC - 1) / kC : 0;
  p.last = seg == live - 1;
  return p;
}

// The CTA's walk once more, its tokens one after the other, by 128 threads with a column of the state each: for inputs with
// infinities or NaN, which the tiles' products multiply by the zeros of the tokens before them too.  (It finds its place
// again by itself: what it would be handed would hold registers through the whole kernel, which took 3 % longer.)
__device__ __noinline__ void walk_tokens(const Walk& w, float* m) {
  using T = __nv_bfloat16;
  const int h = blockIdx.x % w.H, b = blockIdx.x / w.H, c = threadIdx.x, da = w.da;
  const Seq q = seq_of(w.lengths, w.index, b, w.L, w.slots, St{nullptr, 0u});
  const Span sp = span_of(w, blockIdx.y, q.len);
  const long long cells = (long long)da * w.dc, slot = (q.slot * w.H + h) * cells;
  const float g = decay_of(w.log_decay, h), less = expm1f(g);
  float *sa = m + da * kC, *sb = sa + kC;
  if (c < w.dc) {
    const float* local = w.local + (((long long)b * w.H + h) * w.segs + blockIdx.y) * cells;
    const float by = w.init_scale * (w.reverse ? 1.f : power(g, 1));
    for (int r = 0; r < da; ++r)
      m[r * kC + c] = w.segs > 1 ? rd(local + r + (long long)c * da)
                                 : w.init && q.slot >= 0 ? by * rd(w.init + slot + r * w.init_r + c * w.init_c) : 0.f;
  }
  const int n = sp.end - sp.begin;
  // a token's values are on their way while the one before is worked on
  const auto token = [&](int i) { return (long long)(w.reverse ? sp.end - 1 - i : sp.begin + i); };
  T xa, xb, xc;
  const auto load = [&](int i) {
    if (c < da) xa = rd(at_head<T>(w.a, b, h) + token(i) * w.a.row + c), xb = rd(at_head<T>(w.b, b, h) + token(i) * w.b.row + c);
    if (c < w.dc) xc = rd(at_head<T>(w.c, b, h) + token(i) * w.c.row + c);
  };
  load(0);
  for (int i = 0; i < n; ++i) {
    const long long t = token(i);
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (c < da) sa[c] = to_f(xa), sb[c] = to_f(xb);
    const float x = to_f(xc);
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (i + 1 < n) load(i + 1);
    if (c >= w.dc) continue;
    float sum[4] = {};
    const float keep = i == 0 ? 0.f : less;
    const auto rows = [&](auto count, int r0) {
      constexpr int N = decltype(count)::value;
      float v[N];
#pragma unroll
      for (int y = 0; y < N; ++y) v[y] = m[(r0 + y) * kC + c];
#pragma unroll
      for (int y = 0; y < N; ++y) {
        v[y] = fmaf(sb[r0 + y], x, fmaf(v[y], keep, v[y]));
        sum[y & 3] = fmaf(sa[r0 + y], v[y], sum[y & 3]);
      }
#pragma unroll
      for (int y = 0; y < N; ++y) m[(r0 + y) * kC + c] = v[y];
    };
    int r0 = 0;
    for (; r0 + 16 <= da; r0 += 16) rows(std::integral_constant<int, 16>{}, r0);
    for (; r0 < da; ++r0) rows(std::integral_constant<int, 1>{}, r0);
    const float out = w.scale * ((sum[0] + sum[1]) + (sum[2] + sum[3]));
    const long long at = b * w.out_batch + t * w.out_row + h * w.out_head + c;
    if (w.out_f32)
      wr(static_cast<float*>(w.out) + at, out);
    else
      wr(static_cast<T*>(w.out) + at, from_f<T>(out));
  }
  if (sp.last && w.last && q.slot >= 0 && c < w.dc)
    for (int r = 0; r < da; ++r) {
      const float v = m[r * kC + c];
      wr(w.last + slot + r * w.init_r + c * w.init_c, w.last_scale * (w.reverse ? fmaf(v, less, v) : v));
    }
}

// Whether a chunk's sums that the state has not taken up are not finite: those of the walk's last chunk, where no state is
// returned.
template <int DV>
__device__ __noinline__ bool last_lost(const Walk& w, uint32_t o1) {
  const int b = blockIdx.x / w.H;
  const Seq q = seq_of(w.lengths, w.index, b, w.L, w.slots, St{nullptr, 0u});
  const Span sp = span_of(w, blockIdx.y, q.len);
  if (sp.last && w.last && q.slot >= 0) return false;
  const int n = w.reverse ? sp.end - sp.begin : sp.end - sp.begin - kC * (sp.chunks - 1);  // rows of the chunk: that many, or all
  float2 zero = make_float2(0.f, 0.f);  // or NaN
#pragma unroll 1
  for (int c = 0; c < DV; c += 32) {
    uint32_t u[32];
    tmem_ld32(o1 + c, u);
#pragma unroll
    for (int x = 0; x < 16; ++x)
      zero = fma2(make_float2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])), make_float2(0.f, 0.f), zero);
  }
  return (int)threadIdx.x < n && !(zero.x + zero.y == 0.f);
}

// 512 threads: warps 0 to 3 form P and put out O, warps 4 to 7 hold the state (with more registers: 208 a thread of the
// 4 x 128 that the four warpgroups start with), warp 8 brings the tiles, warp 9 issues the products, warps 12 to
// 15 scale the keys.  Every wait is bounded; where one gives up the CTA records a stall,
// waits for its copies and products in flight, frees its tensor memory and leaves.
//
// A later token's weight of 0 times an infinity or NaN is NaN, so outputs before it in its chunk are lost.  Any such value
// leaves the state infinite or NaN in its column for good: the state's warps look once, at the end (warps 0 to 3 at the
// sums of a last chunk that the state does not take up), and warps 0 to 3 then go through the tokens again one by one
// (looking at every chunk's sums, with a call there to form them again, took 4 to 13 % longer; this way
// 0 to 3 %).  The roles lie in the order in which the instruction caches take them best: with the keys behind the state 65536 tokens
// of 16 heads of 64 took 284 us instead of 266, the other cases 1 % less.
template <int DK, int DV, int NK, bool STATE>
__global__ void __launch_bounds__(kThreads, 1) tiles_kernel(const __grid_constant__ Passes ps, s4impl::St st) {
  using R = Room<DK, DV, NK, STATE>;
  static_assert(R::BYTES - 1024 >= 4 * kC * (DK + 2), "shared memory of walk_tokens");
  const Walk& w = ps.walks.w[blockIdx.z];
  const Maps& maps = ps.maps[blockIdx.z];
  extern __shared__ char raw[];
  __shared__ unsigned long long full_a[2], full_b[2], full_c[2], empty_a[2], empty_b[2], empty_c[2];
  __shared__ unsigned long long keys_ready[4], keys_free[4];
  __shared__ unsigned long long s_ready, p_ready, c_clean, d_ready, d_free, m_ready, m_free, o_ready, o_free, idle;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int failed, lost;
  __shared__ __align__(16) float tab[32];
  char* smem = raw + (-s4dev::smem_u32(raw) & 1023);  // (still a shared-memory address to the compiler)
  const int wid = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // (uniform)
  const int h = blockIdx.x % w.H, b = blockIdx.x / w.H, seg = blockIdx.y;
  record_gen(st);
  const Seq q = seq_of(w.lengths, w.index, b, w.L, w.slots, st);
  const Span sp = span_of(w, seg, q.len);
  const float g = decay_of(w.log_decay, h);
  const long long cells = (long long)w.da * w.dc;
  const float* init = w.init && q.slot >= 0 ? w.init + (q.slot * w.H + h) * cells : nullptr;
  float* last = w.last && q.slot >= 0 ? w.last + (q.slot * w.H + h) * cells : nullptr;
  if (!STATE) {
    // padding, in the order of memory
    const int from = q.len > seg * w.seg ? q.len : seg * w.seg, to = (seg + 1) * w.seg < w.L ? (seg + 1) * w.seg : w.L;
    blank_rows<__nv_bfloat16>(w, b, h, 0, w.dc, from, to);
    if (q.len == 0 && last && seg == 0)
      for (int i = threadIdx.x; i < cells; i += kThreads) wr(last + i, init ? rd(init + i) : 0.f);
  }
  if (sp.chunks <= 0 || (STATE && sp.last)) return;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      s4dev::mbar_init(&full_a[i], 1), s4dev::mbar_init(&full_b[i], 1), s4dev::mbar_init(&full_c[i], 1);
      s4dev::mbar_init(&empty_a[i], 1), s4dev::mbar_init(&empty_b[i], STATE ? 4 : 5), s4dev::mbar_init(&empty_c[i], 1);
    }
    for (int i = 0; i < 4; ++i) s4dev::mbar_init(&keys_ready[i], 4), s4dev::mbar_init(&keys_free[i], 1);
    s4dev::mbar_init(&s_ready, 1), s4dev::mbar_init(&p_ready, 4), s4dev::mbar_init(&c_clean, 4);
    s4dev::mbar_init(&d_ready, 1), s4dev::mbar_init(&d_free, 4), s4dev::mbar_init(&m_ready, 4), s4dev::mbar_init(&m_free, 1);
    s4dev::mbar_init(&o_ready, 1), s4dev::mbar_init(&o_free, 4), s4dev::mbar_init(&idle, 1);
    failed = lost = 0;
    s4dev::fence_mbar_init();
  }
  if (threadIdx.x < 32) tab[threadIdx.x] = power(g, threadIdx.x);
  if (wid == 9) tmem_alloc(&tmem_slot, R::COLS);
  fence_before();
  __syncthreads();
  fence_after();
  constexpr uint32_t tmem = 0;  // where an allocation of all the columns begins
  const int limit = ps.limit;
  const auto wait = [&](unsigned long long* bar, unsigned parity) {
    for (int it = 0; it < limit; it += 256) {
      if (s4dev::mbar_wait(bar, parity & 1, limit - it < 256 ? limit - it : 256)) return true;
      if (failed) return false;
    }
    failed = 1;
    return false;
  };
  const auto wait_warp = [&](unsigned long long* bar, unsigned parity) {
    return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
  };
  // two barriers, tested at once
  const auto wait_both = [&](unsigned long long* x, unsigned px, unsigned long long* y, unsigned py) {
    const bool a = s4dev::mbar_wait(x, px & 1, 1), b = s4dev::mbar_wait(y, py & 1, 1);
    return __all_sync(0xffffffffu, (a || wait(x, px)) && (b || wait(y, py))) != 0;
  };
  // chunk k of the walk begins at token `start`
  const auto start_of = [&](int k) { return sp.begin + kC * (w.reverse ? sp.chunks - 1 - k : k); };
  const auto updates = [&](int k) { return STATE || k + 1 < sp.chunks || (sp.last && last != nullptr); };

  int na = 0, nb = 0, nc = 0;  // tiles asked for
  if (wid >= 8 && wid < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (wid == 8 && elected()) {
      for (int k = 0; k < sp.chunks; ++k) {
        const int t = start_of(k), sb = k % R::SB, sc = k % R::SC;
        if (!wait(&empty_b[sb], k / R::SB + 1)) break;
        s4dev::mbar_expect_tx(&full_b[sb], R::TA);
#pragma unroll
        for (int i = 0; i < DK / 64; ++i)
          tma_load_4d(smem + R::B + sb * R::TA + i * 16384, &maps.b, 64 * i, h / w.b.per, t, b, &full_b[sb]);
        ++nb;
        if constexpr (!STATE) {
          const int sa = k % R::SA;
          if (!wait(&empty_a[sa], k / R::SA + 1)) break;
          s4dev::mbar_expect_tx(&full_a[sa], R::TA);
#pragma unroll
          for (int i = 0; i < DK / 64; ++i)
            tma_load_4d(smem + R::A + sa * R::TA + i * 16384, &maps.a, 64 * i, h / w.a.per, t, b, &full_a[sa]);
          ++na;
        }
        if (!wait(&empty_c[sc], k / R::SC + 1)) break;
        s4dev::mbar_expect_tx(&full_c[sc], R::TC);
#pragma unroll
        for (int i = 0; i < DV / 64; ++i)
          tma_load_4d(smem + R::C + sc * R::TC + i * 16384, &maps.c, 64 * i, h / w.c.per, t, b, &full_c[sc]);
        ++nc;
      }
    } else if (wid == 9) {
      // the warp stays together, so that the descriptors are uniform; one lane issues
      constexpr uint32_t kS = instruction(true, false, false, 128, 128), kAM = instruction(true, false, true, 128, DV),
                         kD = instruction(true, true, true, 128, DV), kPC = instruction(true, false, true, 128, DV);
      const uint32_t base = s4dev::smem_u32(smem);
      const uint32_t one = elected();
      int slots = 0, blanked = 0;  // of keys used, chunks that were not full
      for (int k = 0; k < sp.chunks; ++k) {
        const int sb = k % R::SB, sc = k % R::SC;
        const uint64_t dc = tile_desc(base + R::C + sc * R::TC, 16384);
        const uint64_t da = tile_desc(base + R::A + (STATE ? 0 : (k % (R::SA ? R::SA : 1)) * R::TA), 16);
        if constexpr (!STATE) {
          if (!wait_both(&full_b[sb], k / R::SB, &full_a[k % R::SA], k / R::SA)) break;
          fence_after();
          // S: over the width, 64 at a time
          const uint64_t db = tile_desc(base + R::B + sb * R::TA, 16);
#pragma unroll
          for (int i = 0; i < DK / 16; ++i) {
            const uint32_t at = (i / 4 * 16384 + i % 4 * 32) >> 4;
            mma_f16(R::S, da + at, db + at, kS, i > 0, one);
          }
          mma_commit(&s_ready, one);
          mma_commit(&empty_b[sb], one);
        }
        const bool up = updates(k);
        // where a chunk is not full, C's last rows have been blanked
        if (sp.end - start_of(k) < kC && !wait_warp(&c_clean, blanked++)) break;
        if (!(up ? wait_both(&full_c[sc], k / R::SC, &d_free, k + 1) : wait_warp(&full_c[sc], k / R::SC))) break;
        if (up) {
          bool ok = true;
          for (int j = 0; j < kC / kSlot; ++j, ++slots) {
            const int sk = slots % R::SK;
            ok = wait_warp(&keys_ready[sk], slots / R::SK);
            if (!ok) break;
            fence_after();
#pragma unroll
            for (int p = 0; p < NK; ++p) {
              // widths of 64: 64 rows of the state, and the same once more
              const uint64_t dk = tile_desc(base + R::K + (sk * NK + p) * R::TK, DK == 64 ? 0 : kSlot * 128);
#pragma unroll
              for (int i = 0; i < kSlot / 16; ++i)
                mma_f16(R::D, dk + i * (2048 >> 4), dc + (j * (kSlot / 16) + i) * (2048 >> 4), kD, j + p + i > 0, one);
            }
            mma_commit(&keys_free[sk], one);
          }
          if (!ok) break;
          mma_commit(&d_ready, one);
          if (STATE) mma_commit(&empty_c[sc], one);
        }
        if constexpr (!STATE) {
          if (!wait_both(&m_ready, k, &o_free, k + 1)) break;
          fence_after();
          const uint64_t dm = tile_desc(base + R::M, DK * 128);
#pragma unroll
          for (int i = 0; i < DK / 16; ++i)
            mma_f16(R::O2, da + ((i / 4 * 16384 + i % 4 * 32) >> 4), dm + i * (2048 >> 4), kAM, i > 0, one);
          mma_commit(&m_free, one);
          mma_commit(&empty_a[k % R::SA], one);
          if (!wait_warp(&p_ready, k)) break;
          fence_after();
#pragma unroll
          for (int i = 0; i < kC / 16; ++i) mma_tmem_a(R::O1, R::S + i * 8, dc + i * (2048 >> 4), kPC, i > 0, one);
          mma_commit(&o_ready, one);
          mma_commit(&empty_c[sc], one);
        }
      }
    }
  } else if (wid < 4 && !STATE) {
    const auto rows = [&](auto rev) {
      constexpr bool REV = decltype(rev)::value;
      const int i = wid * 32 + lane;
      const uint32_t lanes = tmem + ((uint32_t)wid * 32 << 16);
      const float scale = w.scale;
      const bool f32 = w.out_f32, vec = w.vec, by_map = ps.by_map[blockIdx.z];
      const int dc = w.dc, chunks = sp.chunks;
      const long long row = w.out_row;
      const long long base = b * w.out_batch + h * w.out_head + i * row;
      // The decays within the thread's own 32 columns, the same for every chunk, and words that blank later tokens.
      float2 own[16];
      uint32_t mask[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const int lag = REV ? 2 * x - lane : lane - 2 * x, next = REV ? lag + 1 : lag - 1;
        own[x] = make_float2(tab[lag & 31], tab[next & 31]);
        mask[x] = (lag >= 0 ? 0xffffu : 0u) | (next >= 0 ? 0xffff0000u : 0u);
      }
      for (int k = 0; k < chunks; ++k) {
        const int t = start_of(k), n = sp.end - t < kC ? sp.end - t : kC;
        bool ok = wait_warp(&s_ready, k);
        fence_after();
#pragma unroll 1
        for (int jb = 0; jb < 4 && ok; ++jb) {
          uint32_t p[16];
          if (REV ? jb < wid : jb > wid) {
#pragma unroll
            for (int x = 0; x < 16; ++x) p[x] = 0;
          } else {
            uint32_t s[32];
            tmem_ld32(lanes + R::S + jb * 32, s);
            if (jb == wid) {
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float2 z = mul2(make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])), own[x]);
                p[x] = two_of<__nv_bfloat16>(z.x, z.y) & mask[x];
              }
            } else {
              const float f = power(g, REV ? 32 * jb - i : i - 32 * jb - 31);
              const float2 far = make_float2(f, f);
#pragma unroll
              for (int x = 0; x < 16; x += 2) {
                // the block's nearest column to each of its columns
                const float4 q = *reinterpret_cast<const float4*>(tab + (REV ? 2 * x : 28 - 2 * x));
                const float2 u = mul2(mul2(make_float2(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1])),
                                           REV ? make_float2(q.x, q.y) : make_float2(q.w, q.z)), far);
                const float2 v = mul2(mul2(make_float2(__uint_as_float(s[2 * x + 2]), __uint_as_float(s[2 * x + 3])),
                                           REV ? make_float2(q.z, q.w) : make_float2(q.y, q.x)), far);
                p[x] = two_of<__nv_bfloat16>(u.x, u.y);
                p[x + 1] = two_of<__nv_bfloat16>(v.x, v.y);
              }
            }
            if (REV && 32 * jb + 32 > n) {
              // columns behind the last token hold anything
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                if (32 * jb + 2 * x >= n) p[x] = 0;
                else if (32 * jb + 2 * x + 1 >= n) p[x] &= 0xffffu;
              }
            }
          }
          tmem_st16(lanes + R::S + jb * 16, p);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        fence_before();
        __syncwarp();
        if (lane == 0) arrive(&p_ready);
        ok = ok && wait_warp(&o_ready, k);
        const bool staged = R::STAGED && by_map && n == kC;
        // (the chunk before has been read from the staging rows)
        if (staged && threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        if (!all_of(ok)) break;  // all four warps or none: they meet again below
        fence_after();
        const float e = power(g, REV ? n - 1 - i : i) * scale;
        const float2 ee = make_float2(e, e), sc = make_float2(scale, scale);
        const long long at = base + t * row;
#pragma unroll 1
        for (int c = 0; c < DV; c += 32) {
          uint32_t u[32], v[32];
          tmem_ld32(lanes + R::O1 + c, lanes + R::O2 + c, u, v);
          if (c + 32 == DV) {
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(&o_free);
          }
          if (i >= n || c >= dc) continue;
          float2 f[16];
#pragma unroll
          for (int x = 0; x < 16; ++x)
            f[x] = fma2(make_float2(__uint_as_float(v[2 * x]), __uint_as_float(v[2 * x + 1])), ee,
                        mul2(make_float2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])), sc));
          if (staged) {
#pragma unroll
            for (int x = 0; x < 16; x += 4)
              *reinterpret_cast<uint4*>(smem + R::O + c / 64 * 16384 + i * 128 + ((c % 64 / 8 + x / 4) ^ (i & 7)) * 16) =
                  make_uint4(two_of<__nv_bfloat16>(f[x].x, f[x].y), two_of<__nv_bfloat16>(f[x + 1].x, f[x + 1].y),
                             two_of<__nv_bfloat16>(f[x + 2].x, f[x + 2].y), two_of<__nv_bfloat16>(f[x + 3].x, f[x + 3].y));
          } else {
            put_row(w.out, at + c, dc - c, f32, vec, f);
          }
        }
        if (staged) {
          s4dev::fence_proxy_async();
          asm volatile("bar.sync 1, 128;" ::: "memory");
          if (threadIdx.x == 0) {
            for (int c = 0; c < dc; c += 64) tma_store_4d(&maps.out, smem + R::O + c / 64 * 16384, c, h, t, b);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
      if (R::STAGED && threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    };
    if (w.reverse)
      rows(std::true_type{});
    else
      rows(std::false_type{});
  } else if (wid >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    // The keys of a chunk, scaled: four lanes to a token (odd tokens take the halves of 64 columns in the other
    // order, so that the lanes' packs lie in different banks).
    const int r = (wid - 12) * 32 + lane, chunks = sp.chunks;
    const bool rev = w.reverse;
    int slots = 0;
    bool ok = true;
    for (int k = 0; k < chunks; ++k) {
      const int t = start_of(k), n = sp.end - t < kC ? sp.end - t : kC, sb = k % R::SB, sc = k % R::SC;
      const int less = !STATE && sp.last && k + 1 == chunks && !rev ? 1 : 0;
      if (n < kC) {
        // first of all: the products wait for it before they free the keys' slots
        if (!wait_warp(&full_c[sc], k / R::SC)) break;
        if (r >= n)
#pragma unroll 1
          for (int c = 0; c < DV / 8; ++c)
            *reinterpret_cast<uint4*>(smem + R::C + sc * R::TC + c / 8 * 16384 + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        s4dev::fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive(&c_clean);
      }
      if (!wait_warp(&full_b[sb], k / R::SB)) break;
      if (updates(k)) {
        const int token = r >> 2, quarter = r & 3;
#pragma unroll 1
        for (int j = 0; j < kC; j += kSlot, ++slots) {
          const int sk = slots % R::SK, at = j + token;
          ok = wait_warp(&keys_free[sk], slots / R::SK + 1);
          if (!ok) break;
          const float f = at < n ? power(g, rev ? at + 1 : n - less - at) : 0.f;
          const float2 ff = make_float2(f, f);
          const char* from = smem + R::B + sb * R::TA + at * 128;
          char* to = smem + R::K + sk * NK * R::TK + token * 128;
          const int c0 = ((quarter + 4 * (token & 1)) ^ (token & 7)) * 16, c1 = ((quarter + 4 * (~token & 1)) ^ (token & 7)) * 16;
          uint4 v[DK / 32];
#pragma unroll
          for (int y = 0; y < DK / 32; ++y) v[y] = *reinterpret_cast<const uint4*>(from + y / 2 * 16384 + (y & 1 ? c1 : c0));
#pragma unroll
          for (int y = 0; y < DK / 32; ++y) {
            if (at >= n) v[y] = make_uint4(0, 0, 0, 0);  // behind the last token: anything, NaN too
            const unsigned x[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
            unsigned o[NK][4];
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4) {
              float2 z = mul2(make_float2(__uint_as_float(x[w4] << 16), __uint_as_float(x[w4] & 0xffff0000u)), ff);
#pragma unroll
              for (int p = 0; p < NK; ++p) {
                o[p][w4] = two_of<__nv_bfloat16>(z.x, z.y);
                if (p + 1 < NK)
                  z = fma2(make_float2(__uint_as_float(o[p][w4] << 16), __uint_as_float(o[p][w4] & 0xffff0000u)),
                           make_float2(-1.f, -1.f), z);
              }
            }
#pragma unroll
            for (int p = 0; p < NK; ++p)
              *reinterpret_cast<uint4*>(to + p * R::TK + y / 2 * (kSlot * 128) + (y & 1 ? c1 : c0)) =
                  make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
          }
          s4dev::fence_proxy_async();
          __syncwarp();
          if (lane == 0) arrive(&keys_ready[sk]);
        }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) arrive(&empty_b[sb]);
    }
  } else if (wid >= 4 && wid < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int r = (wid - 4) * 32 + lane;  // a row of the state
    const uint32_t lanes = tmem + ((uint32_t)(wid - 4) * 32 << 16);
    const bool row = r < w.da, rev = w.reverse;
    const int dc = w.dc, chunks = sp.chunks;
    float2 m[DV / 2];  // columns 2 c and 2 c + 1
    float* local = w.local + (((long long)b * w.H + h) * w.segs + seg) * cells;
    {
      // with several segments not from `init`, which may be where the last segment's CTA has put the state on return
      const float by = w.segs > 1 ? 1.f : w.init_scale * (rev ? 1.f : power(g, 1));
      const float* from = STATE || !row ? nullptr : w.segs > 1 ? local + r : init ? init + r * w.init_r : nullptr;
      const long long step = w.segs > 1 ? w.da : w.init_c;
      if (from && step == 1 && dc % 4 == 0 && (uintptr_t)from % 16 == 0) {
#pragma unroll
        for (int c = 0; c < DV / 2; c += 2) {
          float v[4] = {};
          if (2 * c < dc) ld_f<float, 4>(from + 2 * c, 4, true, v);
          m[c] = make_float2(by * v[0], by * v[1]), m[c + 1] = make_float2(by * v[2], by * v[3]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < DV / 2; ++c)
          m[c] = make_float2(from && 2 * c < dc ? by * rd(from + 2 * c * step) : 0.f,
                             from && 2 * c + 1 < dc ? by * rd(from + (2 * c + 1) * step) : 0.f);
      }
    }
    // the state as the right operand of A M: rows of 128 bytes, swizzled
    const auto put = [&] {
      if (r < DK) {
#pragma unroll
        for (int c = 0; c < DV / 2; c += 4) {
          const uint4 v = make_uint4(two_of<__nv_bfloat16>(m[c].x, m[c].y), two_of<__nv_bfloat16>(m[c + 1].x, m[c + 1].y),
                                     two_of<__nv_bfloat16>(m[c + 2].x, m[c + 2].y), two_of<__nv_bfloat16>(m[c + 3].x, m[c + 3].y));
          *reinterpret_cast<uint4*>(smem + R::M + c / 32 * (DK * 128) + r * 128 + ((c % 32 / 4) ^ (r & 7)) * 16) = v;
        }
      }
      s4dev::fence_proxy_async();
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(&m_ready);
    };
    if (!STATE) put();
    for (int k = 0; k < chunks; ++k) {
      if (!updates(k)) break;  // (only the last chunk may have no update)
      const int t = start_of(k), n = sp.end - t < kC ? sp.end - t : kC;
      const int less = !STATE && sp.last && k + 1 == chunks && !rev ? 1 : 0;
      if (!wait_warp(&d_ready, k)) break;
      fence_after();
      const float by = expm1f(g * (float)(n - less));
      const float2 bb = make_float2(by, by);
#pragma unroll
      for (int c = 0; c < DV; c += 32) {
        uint32_t u[32];
        tmem_ld32(lanes + R::D + c, u);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          m[c / 2 + x] = add2(fma2(m[c / 2 + x], bb, m[c / 2 + x]),
                              make_float2(__uint_as_float(u[2 * x]), __uint_as_float(u[2 * x + 1])));
      }
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(&d_free);
      if (!STATE && k + 1 < chunks) {
        if (!wait_warp(&m_free, k)) break;
        put();
      }
    }
    if (!STATE) {
      float2 zero = make_float2(0.f, 0.f);
#pragma unroll
      for (int c = 0; c < DV / 2; ++c) zero = fma2(m[c], make_float2(0.f, 0.f), zero);
      if (!(zero.x + zero.y == 0.f)) lost = 1;
      asm volatile("bar.sync 2, 128;" ::: "memory");
    }
    // (where it is lost the state on return, which may go where the one on entry is, comes from the second walk)
    float* to = STATE ? local + cells + r : last && sp.last ? last + r * w.init_r : nullptr;  // (STATE: the next segment's)
    if (row && to && !failed && (STATE || !lost)) {
      const long long step = STATE ? w.da : w.init_c;
      const float by = STATE ? 1.f : w.last_scale;
      if (step == 1 && dc % 4 == 0 && (uintptr_t)to % 16 == 0) {
#pragma unroll
        for (int c = 0; c < DV / 2; c += 2) {
          const float v[4] = {by * m[c].x, by * m[c].y, by * m[c + 1].x, by * m[c + 1].y};
          if (2 * c < dc) st_f<float, 4>(to + 2 * c, 4, true, v);
        }
      } else {
#pragma unroll
        for (int c = 0; c < DV / 2; ++c) {
          if (2 * c < dc) wr(to + 2 * c * step, by * m[c].x);
          if (2 * c + 1 < dc) wr(to + (2 * c + 1) * step, by * m[c].y);
        }
      }
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  fence_after();
  if (!STATE && wid < 4 && !failed) {
    if (last_lost<DV>(ps.walks.w[blockIdx.z], tmem + ((threadIdx.x & 96) << 16) + R::O1)) lost = 1;
    fence_before();
  }
  if (!STATE) {
    __syncthreads();
    fence_after();
  }
  if (failed) {
    // the copies and products in flight
    if (threadIdx.x == 0 && st.w) s4dev::st_flag(st, s4dev::ST_STALL);
    const auto drain = [](unsigned long long* bar, int issued, int stages) {
      for (int j = issued > stages ? issued - stages : 0; j < issued; ++j)
        s4dev::mbar_wait(&bar[j % stages], (unsigned)(j / stages) & 1);
    };
    drain(full_b, nb, R::SB);
    if constexpr (!STATE) drain(full_a, na, R::SA);
    drain(full_c, nc, R::SC);
    if (wid == 9) {
      mma_commit(&idle, elected());
      s4dev::mbar_wait(&idle, 0);
    }
    fence_before();
    __syncthreads();
    fence_after();
  }
  if (wid == 9) tmem_free(tmem, R::COLS);
  if (!STATE && lost && !failed && threadIdx.x < 128)
    walk_tokens(ps.walks.w[blockIdx.z], reinterpret_cast<float*>(raw + (-s4dev::smem_u32(raw) & 1023)));
}

// ---- host side -----------------------------------------------------------------------------------------
bool stride_ok(long long v, int n) { return n == 1 || (v > 0 && v % 8 == 0 && v < (1ll << 38)); }
bool make_map(CUtensorMap* map, const In& x, int width, int heads, int L, int batch) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const Encode encode = reinterpret_cast<Encode>(map_encoder());
  if (!encode) return false;
  const auto bytes = [&](long long stride, int n) { return (cuuint64_t)(n > 1 ? stride * 2 : (width + 7) / 8 * 16); };
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)batch};
  const cuuint64_t strides[3] = {bytes(x.head, heads), bytes(x.row, L), bytes(x.batch, batch)};
  const cuuint32_t box[4] = {64, 1, kC, 1}, unit[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.p), dims, strides, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DK, int DV, int NK>
cudaError_t launch(const Passes& ps, int passes, St st, cudaStream_t s) {
  const Walk& w = ps.walks.w[0];
  const unsigned walks = (unsigned)(w.batch * w.H);
  if (w.segs > 1) {
    using R = Room<DK, DV, NK, true>;
    constexpr auto state = tiles_kernel<DK, DV, NK, true>;
    allow_shared<state>(R::BYTES);
    {
      s4impl::TimedLaunch tl("linear_attention", s);
      state<<<dim3(walks, w.segs - 1, passes), kThreads, R::BYTES, s>>>(ps, st);
    }
    if (const cudaError_t err = s4impl::launch_join(ps.walks, passes, 2, st, s); err != cudaSuccess) return err;
  }
  using R = Room<DK, DV, NK, false>;
  constexpr auto kernel = tiles_kernel<DK, DV, NK, false>;
  allow_shared<kernel>(R::BYTES);
  s4impl::TimedLaunch tl("linear_attention", s);
  kernel<<<dim3(walks, w.segs, passes), kThreads, R::BYTES, s>>>(ps, st);
  return cudaGetLastError();
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_linear_attention_tiles)
#endif

bool tiles_take(const Walk& w, int dtype) {
  if (dtype != S4_BF16 || w.da > 128 || w.dc > 128) return false;
  const auto ok = [&](const In& x) {
    return (uintptr_t)x.p % 16 == 0 && (x.head == 0 || stride_ok(x.head, w.H / x.per)) && stride_ok(x.row, w.L) &&
           stride_ok(x.batch, w.batch);
  };
  return ok(w.a) && ok(w.b) && ok(w.c);
}

// Segments of a sequence: the number with the least time in chunks one after the other on an SM, a CTA on each.  A
// segment costs about 3 chunks more than its own, one that only leaves its state half as much, two more launches as
// much as 3 chunks.  64 at most, as they are joined one after the other: one head of 128 and 16384 tokens takes 46 us in 64
// segments, 56 in 128; above a million tokens more would pay (2^20: 638 us in 64, 345 in 152).
int tile_segments(long long walks, int L, int passes) {
  const int chunks = (L + kC - 1) / kC;
  const long long sms = num_sms();
  int best = 1;
  double least = 1e300;
  for (int n = 1; n <= chunks && n <= 64; ++n) {
    const int each = (chunks + n - 1) / n, segs = (chunks + each - 1) / each;
    if (segs != n) continue;
    const long long all = (walks * passes * n + sms - 1) / sms, states = (walks * passes * (n - 1) + sms - 1) / sms;
    const double t = (double)all * (each + 3) + (n > 1 ? 0.5 * (double)states * (each + 3) + 3 : 0);
    if (t < least) least = t, best = n;
  }
  return best;
}

cudaError_t launch_tiles(const Walks& ws, int passes, int dtype, St st, cudaStream_t s) {
  static_assert(sizeof(Passes) <= 4096, "kernel parameters");
  Passes ps{};
  ps.limit = wait_limit();
  ps.walks = ws;
  const Walk* w = ws.w;
  const int segs = tile_segments((long long)w->batch * w->H, w->L, passes);
  const int seg = ((w->L + kC - 1) / kC + segs - 1) / segs * kC;
  bool returned = false;
#ifdef S4_BOUNDS_CHECK
  Extents x{};
  x.in(w->log_decay, 4, w->H);
  x.in(w->lengths, 4, w->batch);
  x.in(w->index, 4, w->batch);
#endif
  for (int i = 0; i < passes; ++i) {
    Walk& p = ps.walks.w[i];
    for (In* x : {&p.a, &p.b, &p.c})
      if (x->head == 0) x->per = p.H;  // one head broadcast to all (a map has no strides of 0)
    p.seg = seg, p.segs = (p.L + seg - 1) / seg, p.from_start = true;
    const int e = p.out_f32 ? 4 : 2;
    p.vec = vec_ok(p.out, e, 16, p.out_batch, p.out_row) && vec_ok(p.out, e, 16, p.out_head);
    returned |= p.last != nullptr;
    Maps& m = ps.maps[i];
    if (!make_map(&m.a, p.a, p.da, p.H / p.a.per, p.L, p.batch) || !make_map(&m.b, p.b, p.da, p.H / p.b.per, p.L, p.batch) ||
        !make_map(&m.c, p.c, p.dc, p.H / p.c.per, p.L, p.batch))
      return cudaErrorInvalidValue;
    const In out{p.out, p.out_batch, p.out_row, p.out_head, 1};
    ps.by_map[i] = !p.out_f32 && (uintptr_t)p.out % 16 == 0 && stride_ok(p.out_head, p.H) && stride_ok(p.out_row, p.L) &&
                   stride_ok(p.out_batch, p.batch) && make_map(&m.out, out, p.dc, p.H, p.L, p.batch);
#ifdef S4_BOUNDS_CHECK
    const auto in = [&](const In& r, int d) {
      x.add(r.p, 2, true, false, d, p.batch, r.batch, p.L, r.row, p.H / r.per, r.head);
    };
    in(p.a, p.da), in(p.b, p.da), in(p.c, p.dc);
    x.add(p.out, e, false, true, p.dc, p.batch, p.out_batch, p.L, p.out_row, p.H, p.out_head);
    x.in(p.init, 4, (long long)p.H * p.da * p.dc, p.slots);
    x.out(p.last, 4, (long long)p.H * p.da * p.dc, p.slots);
    if (p.segs > 1) x.scratch(p.local, 4, (long long)p.batch * p.H * p.segs * p.da * p.dc);
#endif
  }
#ifdef S4_BOUNDS_CHECK
  if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
  const auto with = [&](auto dk, auto dv) {
    constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
    return returned ? launch<DK, DV, 3>(ps, passes, st, s) : launch<DK, DV, 2>(ps, passes, st, s);
  };
  constexpr std::integral_constant<int, 64> n64{};
  constexpr std::integral_constant<int, 128> n128{};
  if (w->da <= 64) return w->dc <= 64 ? with(n64, n64) : with(n64, n128);
  return w->dc <= 64 ? with(n128, n64) : with(n128, n128);
}

}  // namespace s4impl
