// Linear attention with a decay for each head, forward and backward.  Every pass of it is one walk
//
//   out_i = scale (sum_{j<=i} e^{g (i-j)} (a_i . b_j) c_j + e^{g i} M^T a_i),   M' = e^{g n} M + sum_j e^{g (n-j)} b_j c_j^T
//
// over the tokens of a sequence in one direction, M being the state that the first of them sees (already
// decayed once): forward (a, b, c) = (q, k, v); the gradients of q (dout, v, k), and from the
// end, with the state's gradient as M, those of k (v, dout, q) and v (k, q, dout).
//
// Here the walks for all types, widths up to 256 and any strides, on warp-wide products; bfloat16 up to widths of
// 128 at aligned strides goes to linear_attention_tiles.cu.  What bounds these is the latency of their
// products and shared memory: 4 x 4096 tokens of 16 heads of 128 in bfloat16 at an odd address 0.88 ms, 2.3 for the three
// walks of a backward pass (tiles: 0.12 and 0.22), in float16 1.7 and 4.4, in fp32 2.1 and 5.5; of 256 in bfloat16 2.3
// and 4.9; gradients of 2 x 333 tokens of 6 heads of 48 and 80 in fp32 73 us.  Outputs of widths above 128 spill 64 to 130
// bytes a thread at 255 registers.
#include "linear_attention.cuh"

namespace {
using namespace s4blk;
using s4impl::In;
using s4impl::Walk;
using s4impl::Walks;

constexpr int kThreads = 128, kCols = 64;  // per CTA: 4 warps, columns of c

// ---- matrix products of 16x8x16 bfloat16 tiles ------------------------------------------------------
__device__ __forceinline__ void ldsm(unsigned (&r)[4], const __nv_bfloat16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(s4dev::smem_u32(p)));
}
__device__ __forceinline__ void ldsm_t(unsigned (&r)[4], const __nv_bfloat16* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(s4dev::smem_u32(p)));
}
__device__ __forceinline__ void mma(float (&d)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two values as NP words of two bfloat16 terms each: a term is what the ones before leave of the
// value, rounded (8 bits each).
template <int NP>
__device__ __forceinline__ void split(float x, float y, unsigned (&w)[NP]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    w[p] = two_of<__nv_bfloat16>(x, y);
    x -= __uint_as_float(w[p] << 16);
    y -= __uint_as_float(w[p] & 0xffff0000u);
  }
}
__device__ __forceinline__ float lo_of(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(unsigned w) { return __uint_as_float(w & 0xffff0000u); }

// Terms of an input: a bfloat16 is itself, a float16 two bfloat16, a float three.
template <typename T>
constexpr int kTerms = std::is_same_v<T, float> ? 3 : std::is_same_v<T, __half> ? 2 : 1;

template <typename T, int D, int C>
constexpr int kWalkBytes = 2 * kTerms<T> * (2 * C * (D + 8) + (C + D) * (kCols + 8));
template <typename T, int D, int C>
constexpr bool kTokensFit = kWalkBytes<T, D, C> >= 4 * (D * (kCols + 2) + kThreads);  // see walk_tokens

// Rows [i0, i0 + n) of the walk, columns [c0, c0 + W) of `width`, as terms in shared memory [terms][C][W + 8].
template <typename T, int W, int C>
__device__ __forceinline__ void load_rows(__nv_bfloat16* s, const T* p, long long row, int first, int step, int n, int width,
                                          bool vec) {
  constexpr int NP = kTerms<T>, PACKS = W / 8;
#pragma unroll 4
  for (int i = threadIdx.x; i < C * PACKS; i += kThreads) {
    const int r = i / PACKS, c = (i % PACKS) * 8;
    Pack<T, 8> v;
    const int have = r < n ? width - c : 0;
    if (have > 0)
      v = ld_pack<T, 8>(p + (long long)(first + step * r) * row + c, have < 8 ? have : 8, vec);
    else
      v.zero();
    __nv_bfloat16* at = s + r * (W + 8) + c;
    if constexpr (NP == 1) {
      *reinterpret_cast<uint4*>(at) = *reinterpret_cast<const uint4*>(v.w);
    } else {
      unsigned w[4][NP];
#pragma unroll
      for (int j = 0; j < 4; ++j) split<NP>(v.get(2 * j), v.get(2 * j + 1), w[j]);
#pragma unroll
      for (int t = 0; t < NP; ++t)
        *reinterpret_cast<uint4*>(at + t * C * (W + 8)) = make_uint4(w[0][t], w[1][t], w[2][t], w[3][t]);
    }
  }
}

// The CTA's walk once more, its tokens one after the other, a column of the state for every two threads: for inputs with
// infinities or NaN, which the products of a chunk multiply by the zeros of the tokens before them too.  (It finds its
// place again by itself: what it would be handed would hold registers through the whole kernel.)
template <typename T>
__device__ __noinline__ void walk_tokens(const Walk& w, float* m) {
  const int nc = (w.dc + kCols - 1) / kCols, c0 = (int)(blockIdx.x % nc) * kCols, h = (int)(blockIdx.x / nc) % w.H;
  const int b = (int)(blockIdx.x / nc) / w.H, seg = blockIdx.y, cols = w.dc - c0 < kCols ? w.dc - c0 : kCols, da = w.da;
  const Seq q = seq_of(w.lengths, w.index, b, w.L, w.slots, St{nullptr, 0u});
  const int begin = seg * w.seg, end = begin + w.seg < q.len ? begin + w.seg : q.len;
  const int c = threadIdx.x % kCols, half = threadIdx.x / kCols;
  const bool column = c < cols;
  const long long cells = (long long)da * w.dc, slot = (q.slot * w.H + h) * cells;
  const float g = decay_of(w.log_decay, h), less = expm1f(g);
  float *sa = m + da * kCols, *sb = sa + da, *part = sb + da;
  if (column) {
    const float* local = w.local + (((long long)b * w.H + h) * w.segs + seg) * cells;
    const float by = w.init_scale * (w.reverse ? 1.f : power(g, 1));
    for (int r = half; r < da; r += 2)
      m[r * kCols + c] = w.segs > 1 ? rd(local + (long long)r * w.dc + c0 + c)
                                    : w.init && q.slot >= 0 ? by * rd(w.init + slot + r * w.init_r + (c0 + c) * w.init_c) : 0.f;
  }
  for (int i = begin; i < end; ++i) {
    const long long t = w.reverse ? q.len - 1 - i : i;
    __syncthreads();
    for (int r = threadIdx.x; r < da; r += kThreads) {
      sa[r] = to_f(rd(at_head<T>(w.a, b, h) + t * w.a.row + r));
      sb[r] = to_f(rd(at_head<T>(w.b, b, h) + t * w.b.row + r));
    }
    __syncthreads();
    float sum = 0.f;
    if (column) {
      const float x = to_f(rd(at_head<T>(w.c, b, h) + t * w.c.row + c0 + c));
      for (int r = half; r < da; r += 2) {
        float v = m[r * kCols + c];
        v = fmaf(sb[r], x, i == begin ? v : fmaf(v, less, v));
        sum = fmaf(sa[r], v, sum);
        m[r * kCols + c] = v;
      }
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    if (!column || half) continue;
    const long long at = b * w.out_batch + t * w.out_row + h * w.out_head + c0 + c;
    sum = w.scale * (part[c] + part[kCols + c]);
    if (w.out_f32)
      wr(static_cast<float*>(w.out) + at, sum);
    else
      wr(static_cast<T*>(w.out) + at, from_f<T>(sum));
  }
  if (end == q.len && w.last && q.slot >= 0 && column)
    for (int r = half; r < da; r += 2) {
      const float v = m[r * kCols + c];
      wr(w.last + slot + r * w.init_r + (c0 + c) * w.init_c, w.last_scale * (w.reverse ? fmaf(v, less, v) : v));
    }
}

// The walk of one sequence, head and 64 columns of c, over one segment of the sequence, in chunks of C
// tokens: the sums over a chunk's own tokens are products of its tiles, those over earlier tokens go
// through M, in registers (warp w has rows w D/4 on).  D: da rounded up.  STATE: only M, from zero, for
// the segments after it.  Where outputs are not finite the walk is made once more, token by token: a later token's
// weight of 0 times an infinity or NaN is NaN.
template <typename T, int D, int C, bool STATE>
__global__ void __launch_bounds__(kThreads) walk_kernel(const __grid_constant__ Walks ws, St st) {
  const Walk& w = ws.w[blockIdx.z];
  constexpr int NP = kTerms<T>, NK = 3;  // terms of inputs, of scaled keys
  constexpr int RW = C / 16, CW = 4 / RW, NT = kCols / 8 / CW;  // warps along tokens and columns, column tiles each
  constexpr int MT = D / 64;                                    // tiles of 16 rows of M per warp
  constexpr int PA = D + 8, PC = kCols + 8, SA = C * PA, SC = C * PC, SM = D * PC;
  extern __shared__ __align__(16) char walk_smem[];
  __nv_bfloat16* sa = reinterpret_cast<__nv_bfloat16*>(walk_smem);
  __nv_bfloat16 *sb = sa + NP * SA, *sc = sb + NP * SA, *sm = sc + NP * SC;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, g4 = lane >> 2, t4 = lane & 3;
  const int nc = (w.dc + kCols - 1) / kCols;
  if (blockIdx.x >= (unsigned)(w.batch * w.H * nc)) return;  // (the other walks have more columns)
  const int c0 = (int)(blockIdx.x % nc) * kCols, h = (int)(blockIdx.x / nc) % w.H, b = (int)(blockIdx.x / nc) / w.H;
  const int seg = blockIdx.y, cols = w.dc - c0 < kCols ? w.dc - c0 : kCols;
  record_gen(st);
  const Seq q = seq_of(w.lengths, w.index, b, w.L, w.slots, st);
  const int begin = seg * w.seg, end = begin + w.seg < q.len ? begin + w.seg : q.len;
  const float g = decay_of(w.log_decay, h);
  const T *pa = at_head<T>(w.a, b, h), *pb = at_head<T>(w.b, b, h), *pc = at_head<T>(w.c, b, h) + c0;

  if (STATE && begin + w.seg >= q.len) return;  // no tokens behind this segment
  if (!STATE) {
    // padding, in the order of memory
    const int from = q.len > begin ? q.len : begin, to = begin + w.seg < w.L ? begin + w.seg : w.L;
    blank_rows<T>(w, b, h, c0, cols, from, to);
  }
  const long long cells = (long long)w.da * w.dc;
  const float* init = w.init && q.slot >= 0 ? w.init + (q.slot * w.H + h) * cells : nullptr;
  float* last = w.last && q.slot >= 0 ? w.last + (q.slot * w.H + h) * cells : nullptr;
  if (!STATE && q.len == 0) {
    if (last && seg == 0)
      for (int i = threadIdx.x; i < w.da * cols; i += kThreads) {
        const long long at = (i / cols) * w.init_r + (c0 + i % cols) * w.init_c;
        wr(last + at, init ? rd(init + at) : 0.f);
      }
    return;
  }
  if (begin >= q.len) return;

  // M: element (row, col) of tile (i, j): rows m0 + 16 i + g4 (+8), columns 8 j + 2 t4 (+1)
  const int m0 = wid * (D / 4);
  float m[MT][8][4];
  const auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = m0 + 16 * i + g4 + (e >> 1) * 8, c = 8 * j + 2 * t4 + (e & 1);
          f(m[i][j][e], r, c, r < w.da && c < cols);
        }
  };
  float* local = w.local + (((long long)b * w.H + h) * w.segs + seg) * cells + c0;
  if (STATE || (w.segs == 1 && !init)) {
    each([&](float& v, int, int, bool) { v = 0.f; });
  } else if (w.segs == 1) {
    const float by = w.init_scale * (w.reverse ? 1.f : power(g, 1));
    each([&](float& v, int r, int c, bool in) { v = in ? by * rd(init + r * w.init_r + (c0 + c) * w.init_c) : 0.f; });
  } else {
    // not from `init`, which may be where the last segment's CTA has put the state on return
    each([&](float& v, int r, int c, bool in) { v = in ? rd(local + (long long)r * w.dc + c) : 0.f; });
  }

  float zero = 0.f;  // or NaN, where an output is not finite
  for (int i0 = begin; i0 < end; i0 += C) {
    const int n = end - i0 < C ? end - i0 : C, first = w.reverse ? q.len - 1 - i0 : i0, step = w.reverse ? -1 : 1;
    const bool at_end = i0 + n >= q.len;
    __syncthreads();
    if (!STATE) {
      load_rows<T, D, C>(sa, pa, w.a.row, first, step, n, w.da, w.vec);
      // the state that this chunk sees
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            unsigned t[NP];
            split<NP>(m[i][j][2 * half], m[i][j][2 * half + 1], t);
            __nv_bfloat16* at = sm + (m0 + 16 * i + g4 + 8 * half) * PC + 8 * j + 2 * t4;
#pragma unroll
            for (int p = 0; p < NP; ++p) *reinterpret_cast<unsigned*>(at + p * SM) = t[p];
          }
    }
    load_rows<T, D, C>(sb, pb, w.b.row, first, step, n, w.da, w.vec);
    load_rows<T, kCols, C>(sc, pc, w.c.row, first, step, n, cols, w.vec);
    __syncthreads();

    if (!STATE) {
      const int r0 = (wid % RW) * 16, n0 = (wid / RW) * (NT * 8);
      if (r0 < n) {
        // In fp32 the pairs of terms below the largest are summed by themselves: the tensor cores cut off what each addition
        // shifts out (in one accumulator outputs are off by 0.8e-6 to 2.2e-6 for widths of 48 to 256, apart by 2e-7 to 4e-7).
        constexpr bool APART = NP == 3;
        float o[NT][4], low[APART ? NT : 1][4];
#pragma unroll
        for (int j = 0; j < NT; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
#pragma unroll
        for (int j = 0; j < (APART ? NT : 1); ++j) low[j][0] = low[j][1] = low[j][2] = low[j][3] = 0.f;
        // a pair's products into two column tiles
        const auto add = [&](int j, const unsigned (&f)[4], const unsigned (&b)[4], bool small) {
          float(&x)[4] = APART && small ? low[APART ? j : 0] : o[j];
          float(&y)[4] = APART && small ? low[APART ? j + 1 : 0] : o[j + 1];
          mma(x, f, b[0], b[1]);
          mma(y, f, b[2], b[3]);
        };
#pragma unroll
        for (int k = 0; k < D; k += 16) {
          unsigned fa[NP][4];
#pragma unroll
          for (int p = 0; p < NP; ++p) ldsm(fa[p], sa + p * SA + (r0 + (lane & 15)) * PA + k + (lane >> 4) * 8);
#pragma unroll
          for (int j = 0; j < NT; j += 2) {
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              unsigned fb[4];
              ldsm_t(fb, sm + p * SM + (k + (lane & 15)) * PC + n0 + 8 * j + (lane >> 4) * 8);
#pragma unroll
              for (int u = 0; u + p < NP; ++u) add(j, fa[u], fb, u + p > 0);
            }
          }
        }
        const int i_lo = r0 + g4, i_hi = i_lo + 8;
        const float d_lo = power(g, i_lo), d_hi = power(g, i_hi);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          o[j][0] *= d_lo, o[j][1] *= d_lo, o[j][2] *= d_hi, o[j][3] *= d_hi;
          if constexpr (APART) low[j][0] *= d_lo, low[j][1] *= d_lo, low[j][2] *= d_hi, low[j][3] *= d_hi;
        }
        for (int j0 = 0; j0 <= r0; j0 += 16) {
          float s[2][4] = {}, s_low[APART ? 2 : 1][4] = {};
#pragma unroll
          for (int k = 0; k < D; k += 16) {
            unsigned fa[NP][4];
#pragma unroll
            for (int p = 0; p < NP; ++p) ldsm(fa[p], sa + p * SA + (r0 + (lane & 15)) * PA + k + (lane >> 4) * 8);
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              unsigned fb[4];
              ldsm(fb, sb + p * SA + (j0 + (lane & 7) + (lane >> 4) * 8) * PA + k + (lane >> 3 & 1) * 8);
#pragma unroll
              for (int u = 0; u + p < NP; ++u) {
                mma(APART && u + p > 0 ? s_low[0] : s[0], fa[u], fb[0], fb[1]);
                mma(APART && u + p > 0 ? s_low[APART ? 1 : 0] : s[1], fa[u], fb[2], fb[3]);
              }
            }
          }
          if (APART) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int y = 0; y < 4; ++y) s[x][y] += s_low[APART ? x : 0][y];
          }
          // the decayed weights as the left operand of the next product
          unsigned fp[NP][4];
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const int lag = i_lo + 8 * half - (j0 + 8 * x + 2 * t4);
              const float u = lag >= 0 ? s[x][2 * half] * power(g, lag) : 0.f;
              const float v = lag >= 1 ? s[x][2 * half + 1] * power(g, lag - 1) : 0.f;
              unsigned t[NP];
              split<NP>(u, v, t);
#pragma unroll
              for (int p = 0; p < NP; ++p) fp[p][2 * x + half] = t[p];
            }
#pragma unroll
          for (int j = 0; j < NT; j += 2)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              unsigned fb[4];
              ldsm_t(fb, sc + p * SC + (j0 + (lane & 15)) * PC + n0 + 8 * j + (lane >> 4) * 8);
#pragma unroll
              for (int u = 0; u + p < NP; ++u) add(j, fp[u], fb, u + p > 0);
            }
        }
        if (APART) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int y = 0; y < 4; ++y) o[j][y] += low[APART ? j : 0][y];
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int i = r0 + g4 + 8 * half;
          if (i >= n) continue;
          const long long at = b * w.out_batch + (long long)(first + step * i) * w.out_row + h * w.out_head + c0;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const int c = n0 + 8 * j + 2 * t4;
            const float v[2] = {w.scale * o[j][2 * half], w.scale * o[j][2 * half + 1]};
            if (c >= cols) continue;
            zero = fmaf(v[0], 0.f, fmaf(v[1], 0.f, zero));
            if (w.out_f32)
              st_f<float, 2>(static_cast<float*>(w.out) + at + c, cols - c, w.vec, v);
            else
              st_f<T, 2>(static_cast<T*>(w.out) + at + c, cols - c, w.vec, v);
          }
        }
      }
      if (at_end ? !last : i0 + n >= end) break;  // nothing needs the state any more
    }

    // M' = e^{g n} M + sum_j e^{g (n - j)} b_j c_j^T; what is kept as the forward pass's state has decayed once less
    const int less = !STATE && at_end && !w.reverse ? 1 : 0;
    // The chunk's part is summed up by itself, the smallest pairs of terms first, and added rounded: the tensor cores cut off
    // what an addition shifts out, always towards zero, and a state that stayed in their accumulators would
    // drift over long sequences (1.5e-5 after 56321 tokens in fp32).
    const float by = expm1f(g * (float)(n - less));
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      float d[8][4];
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j][0] = d[j][1] = d[j][2] = d[j][3] = 0.f;
#pragma unroll 1
      for (int k = 0; k < C / 16; ++k) {
        float f[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int j = 16 * k + 2 * t4 + (x & 1) + (x >> 1) * 8;
          f[x] = power(g, n - less - j < 0 ? 0 : n - less - j);  // (rows from n on are zeros)
        }
        unsigned fa[NK][4];
        unsigned raw[NP][4];
#pragma unroll
        for (int p = 0; p < NP; ++p)
          ldsm_t(raw[p], sb + p * SA + (16 * k + (lane & 7) + (lane >> 4) * 8) * PA + m0 + 16 * i + (lane >> 3 & 1) * 8);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          float u = 0.f, v = 0.f;
#pragma unroll
          for (int p = NP - 1; p >= 0; --p) u += lo_of(raw[p][x]), v += hi_of(raw[p][x]);
          unsigned t[NK];
          split<NK>(u * f[(x >> 1) * 2], v * f[(x >> 1) * 2 + 1], t);
#pragma unroll
          for (int p = 0; p < NK; ++p) fa[p][x] = t[p];
        }
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          unsigned fb[NP][4];
#pragma unroll
          for (int p = 0; p < NP; ++p) ldsm_t(fb[p], sc + p * SC + (16 * k + (lane & 15)) * PC + 8 * j + (lane >> 4) * 8);
#pragma unroll
          for (int sum = NK - 1; sum >= 0; --sum)
#pragma unroll
            for (int p = 0; p < NP && p <= sum; ++p) {
              mma(d[j], fa[sum - p], fb[p][0], fb[p][1]);
              mma(d[j + 1], fa[sum - p], fb[p][2], fb[p][3]);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) m[i][j][e] = fmaf(m[i][j][e], by, m[i][j][e]) + d[j][e];
    }
  }
  if (STATE) {
    float* to = local + cells;  // the next segment's
    each([&](float& v, int r, int c, bool in) {
      if (in) wr(to + (long long)r * w.dc + c, v);
    });
  } else if (__syncthreads_or(!(zero == 0.f))) {
    walk_tokens<T>(ws.w[blockIdx.z], reinterpret_cast<float*>(walk_smem));
  } else if (last && end == q.len) {
    each([&](float& v, int r, int c, bool in) {
      if (in) wr(last + r * w.init_r + (c0 + c) * w.init_c, w.last_scale * v);
    });
  }
}

// What each segment starts from, in their order: slot 0 the state on entry, slot s + 1, which holds what segment s
// adds, that and what comes before.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Walks ws, St st) {
  const Walk& w = ws.w[blockIdx.z];
  const long long cells = (long long)w.da * w.dc, i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int h = blockIdx.y % w.H, b = blockIdx.y / w.H;
  if (i >= cells) return;
  const Seq q = seq_of(w.lengths, w.index, b, w.L, w.slots, st);
  const float g = decay_of(w.log_decay, h), by = expm1f(g * (float)w.seg);
  // counted from the sequence's start, the first segment of a walk from its end is the one that may not be full
  const int part = w.reverse && w.from_start ? q.len - (q.len - 1) / w.seg * w.seg : w.seg;
  const float by_first = expm1f(g * (float)part);
  float v = 0.f;
  if (w.init && q.slot >= 0)
    v = w.init_scale * (w.reverse ? 1.f : power(g, 1)) *
        rd(w.init + (q.slot * w.H + h) * cells + (w.from_start ? i % w.da : i / w.dc) * w.init_r +
           (w.from_start ? i / w.da : i % w.dc) * w.init_c);
  float* p = w.local + ((long long)b * w.H + h) * w.segs * cells + i;
  wr(p, v);
  for (int s = 1; s * w.seg < q.len; ++s) {
    p += cells;
    v = fmaf(v, s == 1 ? by_first : by, v) + rd(p);
    wr(p, v);
  }
}

// Gradients of shared heads: part [batch][L][H][d], summed over each group's heads in their order.
struct Shared {
  const float* part;
  void* out;
  long long batch, row, head;
  int d;
};
template <typename T>
__global__ void __launch_bounds__(256) group_sum_kernel(Shared k, Shared v, int batch, int L, int H, int G) {
  const Shared& x = blockIdx.y ? v : k;
  const long long n = (long long)batch * L * G * x.d, each = H / G;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int c = (int)(i % x.d), gr = (int)(i / x.d % G);
    const long long token = i / x.d / G;
    const float* p = x.part + (token * H + gr * each) * x.d + c;
    float v = 0.f;
    for (int j = 0; j < each; ++j) v += rd(p + (long long)j * x.d);
    wr(static_cast<T*>(x.out) + (token / L) * x.batch + (token % L) * x.row + gr * x.head + c, from_f<T>(v));
  }
}

// ---- one token -----------------------------------------------------------------------------------
// The state is read and written once, everything else is small: the bound is memory.  A CTA has some
// columns of one head's state, a thread V neighbouring ones of every RG-th row; the sums over rows
// meet in shared memory.  128 sequences of 32 heads of 128 x 128: 81 us (5.8 TB/s), with 8 rows on their way 91.
template <typename T, int V>
__global__ void __launch_bounds__(256) step_kernel(s4_linear_attention_args a, int lanes, int blocks, St st) {
  __shared__ float sums[256][V];
  __shared__ float sq[256], sk[256];
  const int cb = blockIdx.x % blocks, h = (int)(blockIdx.x / blocks) % a.H, b = (int)(blockIdx.x / blocks) / a.H;
  record_gen(st);
  const Seq q = seq_of(a.lengths, a.index, b, 1, a.slots, st);
  const int lane = threadIdx.x % lanes, rg = threadIdx.x / lanes, RG = 256 / lanes, c = (cb * lanes + lane) * V;
  T* o = static_cast<T*>(a.o.p) + b * a.o.batch + h * a.o.head;
  const long long at = (q.slot < 0 ? 0 : q.slot * a.H + h) * a.K * a.V;
  const float* s = a.state && q.slot >= 0 ? a.state + at : nullptr;
  float* to = a.state_out && q.slot >= 0 ? a.state_out + at : nullptr;
  if (q.len == 0) {
    if (c < a.V) {
      if (rg == 0)
        for (int j = 0; j < V; ++j) wr(o + c + j, from_f<T>(0.f));
      if (to && (to != s))
        for (int r = rg; r < a.K; r += RG) {
          float v[V] = {};
          if (s) ld_f<float, V>(s + (long long)r * a.V + c, V, true, v);
          st_f<float, V>(to + (long long)r * a.V + c, V, true, v);
        }
    }
    return;
  }
  const int kv = h / (a.H / a.G);
  const T* pq = static_cast<const T*>(a.q.p) + b * a.q.batch + h * a.q.head;
  const T* pk = static_cast<const T*>(a.k.p) + b * a.k.batch + kv * a.k.head;
  if (threadIdx.x < a.K) {
    sq[threadIdx.x] = to_f(rd(pq + threadIdx.x)) * a.scale;
    sk[threadIdx.x] = to_f(rd(pk + threadIdx.x));
  }
  const float by = expm1f(decay_of(a.log_decay, h));
  float v[V], sum[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    sum[j] = 0.f;
    v[j] = c < a.V ? to_f(rd(static_cast<const T*>(a.v.p) + b * a.v.batch + kv * a.v.head + c + j)) : 0.f;
  }
  __syncthreads();
  if (c < a.V) {
    // 16 rows are on their way at once
    constexpr int N = 16;
    for (int r0 = rg; r0 < a.K; r0 += N * RG) {
      Pack<float, V> x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = r0 + i * RG;
        if (s && r < a.K)
          x[i] = ld_whole<float, V>(s + (long long)r * a.V + c);
        else
          x[i].zero();
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = r0 + i * RG;
        if (r >= a.K) continue;
        float u[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float old = x[i].get(j);
          u[j] = fmaf(sk[r], v[j], fmaf(old, by, old));
          sum[j] = fmaf(sq[r], u[j], sum[j]);
        }
        if (to) st_whole<float, V>(to + (long long)r * a.V + c, u);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) sums[threadIdx.x][j] = sum[j];
  __syncthreads();
  if (rg != 0 || c >= a.V) return;
  for (int r = 1; r < RG; ++r)
#pragma unroll
    for (int j = 0; j < V; ++j) sum[j] += sums[r * lanes + lane][j];
#pragma unroll
  for (int j = 0; j < V; ++j) wr(o + c + j, from_f<T>(sum[j]));
}

template <typename T>
cudaError_t step_t(const s4_linear_attention_args& a, St st, cudaStream_t s) {
  const bool wide = a.V % 4 == 0 && vec_ok(a.state, 4, 16) && vec_ok(a.state_out, 4, 16);
  const int V = wide ? 4 : 1, packs = a.V / V;
  // Columns are shared out until every SM has a few CTAs, in blocks of whole sectors at least.
  int lanes = 1;
  while (lanes < packs && lanes < 64) lanes *= 2;
  const long long heads = (long long)a.batch * a.H;
  while (lanes * V > 8 && heads * ((packs + lanes - 1) / lanes) < 4ll * s4impl::num_sms()) lanes /= 2;
  const int blocks = (packs + lanes - 1) / lanes;
  s4impl::TimedLaunch tl("linear_attention", s);
  if (wide)
    step_kernel<T, 4><<<(unsigned)(heads * blocks), 256, 0, s>>>(a, lanes, blocks, st);
  else
    step_kernel<T, 1><<<(unsigned)(heads * blocks), 256, 0, s>>>(a, lanes, blocks, st);
  return cudaGetLastError();
}

// ---- host side -----------------------------------------------------------------------------------
// Segments of a sequence: as many as give each SM three CTAs, of 64 tokens or more.
int segments(long long walks, int L) {
  const long long want = (3ll * s4impl::num_sms() + walks - 1) / walks, most = (L + 63) / 64;
  const long long n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n);
}
int segment_tokens(int L, int segs) { return ((L + segs - 1) / segs + 63) / 64 * 64; }
size_t local_bytes(int batch, int L, int H, int da, int dc) {
  int segs = segments((long long)batch * H, L);
  for (int passes = 1; passes <= 3; ++passes) {  // whichever kernels the strides allow
    const int n = da <= 128 && dc <= 128 ? s4impl::tile_segments((long long)batch * H, L, passes) : 1;
    segs = n > segs ? n : segs;
  }
  return s4impl::section(segs == 1 ? 0 : sizeof(float) * (size_t)batch * H * segs * da * dc);
}

#ifdef S4_BOUNDS_CHECK
cudaError_t set_walk_extents(const Walks& ws, int n, int e, cudaStream_t s) {
  s4impl::Extents x{};
  x.in(ws.w[0].log_decay, 4, ws.w[0].H);
  x.in(ws.w[0].lengths, 4, ws.w[0].batch);
  x.in(ws.w[0].index, 4, ws.w[0].batch);
  for (int i = 0; i < n; ++i) {
    const Walk& w = ws.w[i];
    const auto add = [&](const In& r, int d) {
      x.add(r.p, e, true, false, d, w.batch, r.batch, w.L, r.row, (w.H + r.per - 1) / r.per, r.head);
    };
    add(w.a, w.da), add(w.b, w.da), add(w.c, w.dc);
    x.add(w.out, w.out_f32 ? 4 : e, false, true, w.dc, w.batch, w.out_batch, w.L, w.out_row, w.H, w.out_head);
    x.in(w.init, 4, (long long)w.H * w.da * w.dc, w.slots);
    x.out(w.last, 4, (long long)w.H * w.da * w.dc, w.slots);
    if (w.segs > 1) x.scratch(w.local, 4, (long long)w.batch * w.H * w.segs * w.da * w.dc);
  }
  return set_extents(x, s);
}
#endif

template <typename T, int D>
cudaError_t walk_d(const Walks& ws, int n, St st, cudaStream_t s) {
  constexpr int C = kTerms<T> == 3 ? 32 : 64, bytes = kWalkBytes<T, D, C>;
  unsigned walks = 0;
  for (int i = 0; i < n; ++i) {
    const unsigned own = (unsigned)((long long)ws.w[i].batch * ws.w[i].H * ((ws.w[i].dc + kCols - 1) / kCols));
    walks = own > walks ? own : walks;
  }
  static_assert(kTokensFit<T, D, C>, "shared memory");
  constexpr auto kernel = walk_kernel<T, D, C, false>;
  allow_shared<kernel>(bytes);
  const int segs = ws.w[0].segs;
  if (segs > 1) {
    constexpr auto state = walk_kernel<T, D, C, true>;
    allow_shared<state>(bytes);
    {
      s4impl::TimedLaunch tl("linear_attention", s);
      state<<<dim3(walks, segs - 1, n), kThreads, bytes, s>>>(ws, st);
    }
    if (const cudaError_t err = s4impl::launch_join(ws, n, (int)sizeof(T), st, s); err != cudaSuccess) return err;
  }
  s4impl::TimedLaunch tl("linear_attention", s);
  kernel<<<dim3(walks, segs, n), kThreads, bytes, s>>>(ws, st);
  return cudaGetLastError();
}
// n walks over the same sequences and heads, in one launch.
template <typename T>
cudaError_t walk_t(Walks ws, int n, St st, cudaStream_t s) {
  constexpr int code = std::is_same_v<T, float> ? S4_F32 : std::is_same_v<T, __half> ? S4_F16 : S4_BF16;
  bool tiles = true;
  for (int i = 0; i < n; ++i)
    tiles = tiles && s4impl::tiles_take(ws.w[i], code) && (ws.w[i].da <= 64) == (ws.w[0].da <= 64) &&
            (ws.w[i].dc <= 64) == (ws.w[0].dc <= 64);
  if (tiles) return s4impl::launch_tiles(ws, n, code, st, s);
  int most = 0, least_cols = ws.w[0].dc;
  for (int i = 0; i < n; ++i) {
    most = ws.w[i].da > most ? ws.w[i].da : most;
    least_cols = ws.w[i].dc < least_cols ? ws.w[i].dc : least_cols;
  }
  const int want = segments((long long)n * ws.w[0].batch * ws.w[0].H * ((least_cols + kCols - 1) / kCols), ws.w[0].L);
  for (int i = 0; i < n; ++i) {
    Walk& w = ws.w[i];
    w.seg = segment_tokens(w.L, want);
    w.segs = (w.L + w.seg - 1) / w.seg;
    const int e = sizeof(T), eo = w.out_f32 ? 4 : e;
    const auto ok = [&](const In& x) { return vec_ok(x.p, e, 16, x.batch, x.row) && vec_ok(x.p, e, 16, x.head); };
    w.vec = ok(w.a) && ok(w.b) && ok(w.c) && vec_ok(w.out, eo, 2 * eo, w.out_batch, w.out_row) &&
            vec_ok(w.out, eo, 2 * eo, w.out_head);
  }
#ifdef S4_BOUNDS_CHECK
  if (const cudaError_t err = set_walk_extents(ws, n, sizeof(T), s); err != cudaSuccess) return err;
#endif
  if (most <= 64) return walk_d<T, 64>(ws, n, st, s);
  return most <= 128 ? walk_d<T, 128>(ws, n, st, s) : walk_d<T, 256>(ws, n, st, s);
}

In in_of(const s4_heads& r, int per) { return {r.p, r.batch, r.row, r.head, per}; }

template <typename T>
cudaError_t fwd_t(const s4_linear_attention_args& a, St st, cudaStream_t s) {
  if (a.L == 1) {
#ifdef S4_BOUNDS_CHECK
    s4impl::Extents x{};
    const int e = sizeof(T);
    x.add(a.q.p, e, true, false, a.K, a.batch, a.q.batch, a.H, a.q.head);
    x.add(a.k.p, e, true, false, a.K, a.batch, a.k.batch, a.G, a.k.head);
    x.add(a.v.p, e, true, false, a.V, a.batch, a.v.batch, a.G, a.v.head);
    x.add(a.o.p, e, false, true, a.V, a.batch, a.o.batch, a.H, a.o.head);
    x.in(a.log_decay, 4, a.H);
    x.in(a.lengths, 4, a.batch);
    x.in(a.index, 4, a.batch);
    x.in(a.state, 4, (long long)a.H * a.K * a.V, a.slots);
    x.out(a.state_out, 4, (long long)a.H * a.K * a.V, a.slots);
    if (const cudaError_t err = set_extents(x, s); err != cudaSuccess) return err;
#endif
    return step_t<T>(a, st, s);
  }
  Walks ws{};
  Walk& w = ws.w[0];
  w.a = in_of(a.q, 1), w.b = in_of(a.k, a.H / a.G), w.c = in_of(a.v, a.H / a.G);
  w.out = a.o.p, w.out_batch = a.o.batch, w.out_row = a.o.row, w.out_head = a.o.head;
  w.log_decay = a.log_decay, w.lengths = a.lengths, w.index = a.index;
  w.init = a.state, w.last = a.state_out, w.init_r = a.V, w.init_c = 1;
  w.local = reinterpret_cast<float*>(static_cast<char*>(a.ws) + s4impl::kStatusBytes);
  w.scale = a.scale, w.init_scale = w.last_scale = 1.f;
  w.batch = a.batch, w.L = a.L, w.H = a.H, w.da = a.K, w.dc = a.V, w.slots = a.slots;
  return walk_t<T>(ws, 1, st, s);
}

template <typename T>
cudaError_t bwd_t(const s4_linear_attention_bwd_args& a, St st, cudaStream_t s) {
  constexpr int code = std::is_same_v<T, float> ? S4_F32 : std::is_same_v<T, __half> ? S4_F16 : S4_BF16;
  const int each = a.H / a.G;
  char* at = static_cast<char*>(a.ws) + s4impl::kStatusBytes;
  const auto take = [&](size_t bytes) {
    float* p = reinterpret_cast<float*>(at);
    at += bytes;
    return p;
  };
  Walks ws{};
  // dk and dv first: they go through the same tokens in the same order, so what one reads the other finds in the L2
  Walk &dk = ws.w[0], &dv = ws.w[1], &dq = ws.w[2];
  for (Walk& x : ws.w) {
    x.log_decay = a.log_decay, x.lengths = a.lengths;
    x.scale = a.scale, x.last_scale = a.scale;
    x.batch = a.batch, x.L = a.L, x.H = a.H, x.slots = a.batch;
  }
  // dk: from the end over (v, dout, q), the state transposed
  dk.a = in_of(a.v, each), dk.b = in_of(a.dout, 1), dk.c = in_of(a.q, 1);
  dk.da = a.V, dk.dc = a.K, dk.init = a.dstate, dk.init_r = 1, dk.init_c = a.V;
  // dv: from the end over (k, q, dout); it leaves the state's gradient
  dv.a = in_of(a.k, each), dv.b = in_of(a.q, 1), dv.c = in_of(a.dout, 1);
  dv.da = a.K, dv.dc = a.V, dv.init = a.dstate, dv.init_r = a.V, dv.init_c = 1, dv.last = a.dstate0;
  // dq: forward over (dout, v, k), the state transposed
  dq.a = in_of(a.dout, 1), dq.b = in_of(a.v, each), dq.c = in_of(a.k, each);
  dq.out = a.dq.p, dq.out_batch = a.dq.batch, dq.out_row = a.dq.row, dq.out_head = a.dq.head;
  dq.da = a.V, dq.dc = a.K, dq.init = a.state0, dq.init_r = 1, dq.init_c = a.V, dq.init_scale = 1.f;
  Shared shared[2];
  for (int i = 0; i < 3; ++i) {
    Walk& w = ws.w[i];
    w.local = take(local_bytes(a.batch, a.L, a.H, w.da, w.dc));
    if (i == 2) continue;
    const s4_heads_out& out = i == 0 ? a.dk : a.dv;
    const int d = w.dc;
    w.reverse = true, w.init_scale = 1.f / a.scale;
    if (each > 1) {
      float* part = take(s4impl::section(sizeof(float) * (size_t)a.batch * a.L * a.H * d));
      w.out = part, w.out_f32 = true, w.out_head = d, w.out_row = (long long)a.H * d, w.out_batch = w.out_row * a.L;
      shared[i] = {part, out.p, out.batch, out.row, out.head, d};
    } else {
      w.out = out.p, w.out_batch = out.batch, w.out_row = out.row, w.out_head = out.head;
    }
  }
  // All in one launch where their tiles have one shape, or where all segments of 64 tokens of all walks fit the SMs, a CTA each (of
  // widths up to 128 two, one after the other): it then saves launches; else the narrower walks are better off with tiles of
  // their own.  48 and 80 channels in fp32: 8 heads of 64 tokens (32 CTAs) 21 us in one, 34 in two launches; 12 of 333
  // (288) 68 and 63 in a captured graph, 77 and 80 in a stream; 8 of 2000 (1024) 209 and 163, of 16000 1781 and 1172.  40
  // and 256 channels: 4 heads of 333 tokens (144) 61 and 85, 8 (288) 111 and 87.
  const auto size = [](int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; };
  const auto columns = [](int d) { return (d + kCols - 1) / kCols; };
  const long long ctas = (long long)a.batch * a.H * (2 * columns(a.K) + columns(a.V)) * ((a.L + 63) / 64);
  const long long fit = (a.K > 128 || a.V > 128 ? 1ll : 2ll) * s4impl::num_sms();
  cudaError_t err;
  if (size(a.K) == size(a.V) || (!s4impl::tiles_take(dk, code) && ctas <= fit)) {
    err = walk_t<T>(ws, 3, st, s);
  } else {
    Walks two = ws, one{};
    two.w[1] = dq;
    one.w[0] = dv;
    err = walk_t<T>(two, 2, st, s);
    if (err == cudaSuccess) err = walk_t<T>(one, 1, st, s);
  }
  if (err != cudaSuccess || each == 1) return err;
#ifdef S4_BOUNDS_CHECK
  s4impl::Extents x{};
  for (int i = 0; i < 2; ++i) {
    x.in(shared[i].part, 4, (long long)a.batch * a.L * a.H * shared[i].d);
    x.add(shared[i].out, sizeof(T), false, true, shared[i].d, a.batch, shared[i].batch, a.L, shared[i].row, a.G, shared[i].head);
  }
  if (const cudaError_t e = set_extents(x, s); e != cudaSuccess) return e;
#endif
  const long long n = ((long long)a.batch * a.L * a.G * (a.K > a.V ? a.K : a.V) + 255) / 256, most = 16ll * s4impl::num_sms();
  s4impl::TimedLaunch tl("linear_attention", s);
  group_sum_kernel<T><<<dim3((unsigned)(n < most ? n : most), 2), 256, 0, s>>>(shared[0], shared[1], a.batch, a.L, a.H, a.G);
  return cudaGetLastError();
}

}  // namespace

namespace s4impl {

#ifdef S4_BOUNDS_CHECK
S4_OOB_COUNTER(oob_linear_attention)
#endif

size_t linear_attention_scratch(int batch, int L, int H, int K, int V) {
  return L == 1 ? 0 : local_bytes(batch, L, H, K, V);
}

cudaError_t launch_join(const Walks& ws, int n, int e, St st, cudaStream_t s) {
#ifdef S4_BOUNDS_CHECK
  if (const cudaError_t err = set_walk_extents(ws, n, e, s); err != cudaSuccess) return err;
#endif
  s4impl::TimedLaunch tl("linear_attention", s);
  const Walk& w = ws.w[0];  // (all have as many cells)
  join_kernel<<<dim3((unsigned)((w.da * w.dc + 255) / 256), w.batch * w.H, n), 256, 0, s>>>(ws, st);
  return cudaGetLastError();
}

cudaError_t launch_linear_attention(const s4_linear_attention_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return fwd_t<float>(a, st, s);
  return a.dtype == S4_BF16 ? fwd_t<__nv_bfloat16>(a, st, s) : fwd_t<__half>(a, st, s);
}

size_t linear_attention_bwd_scratch(int batch, int L, int H, int G, int K, int V) {
  const size_t each = sizeof(float) * (size_t)batch * L * H, part = H == G ? 0 : section(each * K) + section(each * V);
  return 2 * local_bytes(batch, L, H, V, K) + local_bytes(batch, L, H, K, V) + part;
}

cudaError_t launch_linear_attention_bwd(const s4_linear_attention_bwd_args& a, St st, cudaStream_t s) {
  if (a.dtype == S4_F32) return bwd_t<float>(a, st, s);
  return a.dtype == S4_BF16 ? bwd_t<__nv_bfloat16>(a, st, s) : bwd_t<__half>(a, st, s);
}

}  // namespace s4impl
