// The walk that every pass of linear attention is (see linear_attention.cu), as its kernels take it.
#pragma once
#include "s4_block.cuh"
#include "s4_sequence.h"

namespace s4impl {

// One of a walk's inputs: [batch][L][heads][width], head h of the walk reads head h / per.
struct In {
  const void* p;
  long long batch, row, head;
  int per;
};
struct Walk {
  In a, b, c;
  void* out;                  // of the activations' type, or fp32 (out_f32)
  long long out_batch, out_row, out_head;
  const float* log_decay;
  const int *lengths, *index;
  const float* init;          // [slots][heads][...] state on entry, element (r, c) at r init_r + c init_c
  float* last;                // where the state on return goes, laid out the same
  float* local;               // [batch][heads][segs][da][dc], with several segments: what each starts from (from_start:
                              // [dc][da], as the threads with a row each have it)
  long long init_r, init_c;
  float scale, init_scale, last_scale;
  int batch, L, H, da, dc, slots, segs, seg;
  bool reverse, out_f32, vec;
  bool from_start;            // segments and chunks are counted from the sequence's first token (else from the walk's)
};

// The walks of one launch.
struct Walks {
  Walk w[3];
};

// Walks on the fifth-generation tensor cores (linear_attention_tiles.cu): bfloat16, widths up to 128, strides that a
// tensor map can have.
bool tiles_take(const Walk& w, int dtype);
int tile_segments(long long walks, int L, int passes);
cudaError_t launch_tiles(const Walks& ws, int passes, int dtype, St st, cudaStream_t s);
cudaError_t launch_join(const Walks& ws, int n, int e, St st, cudaStream_t s);  // (e: bytes of an element)

}  // namespace s4impl

namespace {
using namespace s4blk;

__device__ __forceinline__ float decay_of(const float* log_decay, int h) {
  const float g = rd(log_decay + h);
  return g < -1e30f ? -1e30f : g;  // -infinity times no tokens is no decay
}
__device__ __forceinline__ float power(float g, int n) { return ex2(g * kLog2e * (float)n); }

// Zeros for tokens [from, to), columns [c0, c0 + cols) of a head's outputs: a warp per row.
template <typename T>
__device__ __forceinline__ void blank_rows(const s4impl::Walk& w, int b, int h, int c0, int cols, int from, int to) {
  const int lane = threadIdx.x & 31, e = w.out_f32 ? 4 : (int)sizeof(T);
  for (int t = from + (int)(threadIdx.x >> 5); t < to; t += (int)(blockDim.x >> 5)) {
    char* row = static_cast<char*>(w.out) + (b * w.out_batch + (long long)t * w.out_row + h * w.out_head + c0) * e;
    if ((uintptr_t)row % 16 == 0 && cols * e % 16 == 0) {
      for (int c = lane * 16; c < cols * e; c += 512)
        if (touch(row + c, 16, 16, true)) *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
    } else if (e == 4) {
      for (int c = lane; c < cols; c += 32) wr(reinterpret_cast<float*>(row) + c, 0.f);
    } else {
      for (int c = lane; c < cols; c += 32) wr(reinterpret_cast<unsigned short*>(row) + c, (unsigned short)0);
    }
  }
}

template <typename T>
__device__ __forceinline__ const T* at_head(const s4impl::In& x, int b, int h) {
  return static_cast<const T*>(x.p) + b * x.batch + (long long)(h / x.per) * x.head;
}

}  // namespace
