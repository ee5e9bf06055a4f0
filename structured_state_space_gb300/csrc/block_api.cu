// C ABI of the selective block's operators (declared in include/s4.h): argument checks
// on the host, then the launches on the caller's stream.
#include <limits.h>
#include <stdint.h>

#include "s4.h"
#include "s4_block.h"

namespace {

constexpr int kMaxBatch = 65535;
constexpr int kMaxLen = 1 << 24;
constexpr int kMaxChannels = 65536;
constexpr int kMaxNormChannels = 16384;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool sizes_ok(int batch, int L, int H) {
  return batch >= 1 && batch <= kMaxBatch && L >= 1 && L <= kMaxLen && H >= 1 && H <= kMaxChannels;
}
// A strided array: present, aligned to its elements, strides not negative.
template <typename Rows>
bool rows_ok(const Rows& r, int dtype) {
  return r.p && aligned(r.p, s4impl::dtype_bytes(dtype)) && r.batch >= 0 && r.row >= 0;
}
bool scan_sizes_ok(int batch, int L, int H, int N, int G) {
  return sizes_ok(batch, L, H) && N >= 1 && N <= 256 && G >= 1 && G <= H && H % G == 0;
}
s4_status ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && aligned(ws, 256) && bytes >= need ? S4_OK : S4_ERR_WORKSPACE;
}
s4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? S4_OK : S4_ERR_CUDA; }

}  // namespace

extern "C" {

s4_status s4_short_conv_fwd(const s4_short_conv_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || !sizes_ok(a->batch, a->L, a->H) || a->W < 2 || a->W > 8)
    return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype);
  if (!rows_ok(a->x, a->dtype) || !rows_ok(a->y, a->dtype) || !a->w || !aligned(a->w, 4) || !aligned(a->bias, 4) ||
      !aligned(a->lengths, 4) || !aligned(a->index, 4) || !aligned(a->state, e) || !aligned(a->state_out, e))
    return S4_ERR_INVALID_ARG;
  if ((a->state || a->state_out) && (a->slots < 1 || (!a->index && a->slots < a->batch))) return S4_ERR_INVALID_ARG;
  // in place: only single tokens (else an output's neighbours still need its input), each at its own address
  if (a->y.p == a->x.p && (a->L > 1 || (a->batch > 1 && a->y.batch != a->x.batch))) return S4_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st{nullptr, 0u};
  if (a->ws) {
    const s4_status w = ws_ok(a->ws, a->ws_bytes, s4impl::kStatusBytes);
    if (w != S4_OK) return w;
    bool chain;
    if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  }
  return cuda_status(s4impl::launch_short_conv(*a, st, s));
}

size_t s4_short_conv_bwd_workspace_bytes(int batch, int L, int H, int W) {
  if (!sizes_ok(batch, L, H) || W < 2 || W > 8) return 0;
  return s4impl::kStatusBytes + s4impl::align256(s4impl::short_conv_bwd_scratch(batch, L, H, W));
}

s4_status s4_short_conv_bwd(const s4_short_conv_bwd_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || !sizes_ok(a->batch, a->L, a->H) || a->W < 2 || a->W > 8)
    return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype);
  if (!rows_ok(a->x, a->dtype) || !rows_ok(a->dy, a->dtype) || !rows_ok(a->dx, a->dtype) || !a->w || !a->dw ||
      !aligned(a->w, 4) || !aligned(a->dw, 4) || !aligned(a->bias, 4) || !aligned(a->dbias, 4) ||
      !aligned(a->lengths, 4) || !aligned(a->state0, e) || !aligned(a->dstate, e) || !aligned(a->dstate0, e))
    return S4_ERR_INVALID_ARG;
  if ((a->dstate0 && a->dstate0 == a->dstate) || a->dx.p == a->x.p || a->dx.p == a->dy.p) return S4_ERR_INVALID_ARG;
  const s4_status w = ws_ok(a->ws, a->ws_bytes, s4_short_conv_bwd_workspace_bytes(a->batch, a->L, a->H, a->W));
  if (w != S4_OK) return w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st;
  bool chain;
  if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  return cuda_status(s4impl::launch_short_conv_bwd(*a, st, s));
}

size_t s4_selective_scan_workspace_bytes(int batch, int L, int H, int N, int G) {
  if (!scan_sizes_ok(batch, L, H, N, G)) return 0;
  return s4impl::kStatusBytes + s4impl::align256(s4impl::selective_scratch(batch, L, H, N, G));
}

s4_status s4_selective_scan_fwd(const s4_selective_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || !scan_sizes_ok(a->batch, a->L, a->H, a->N, a->G)) return S4_ERR_INVALID_ARG;
  if (!rows_ok(a->x, a->dtype) || !rows_ok(a->dt, a->dtype) || (a->z.p && !rows_ok(a->z, a->dtype)) ||
      !rows_ok(a->B, a->dtype) || !rows_ok(a->C, a->dtype) || !rows_ok(a->y, a->dtype) || a->B_group < 0 ||
      a->C_group < 0 || !a->A || !aligned(a->A, 4) || !aligned(a->D, 4) || !aligned(a->dt_bias, 4) ||
      !aligned(a->lengths, 4) || !aligned(a->index, 4) || !aligned(a->state, 4) || !aligned(a->state_out, 4))
    return S4_ERR_INVALID_ARG;
  if ((a->state || a->state_out) && (a->slots < 1 || (!a->index && a->slots < a->batch))) return S4_ERR_INVALID_ARG;
  const size_t need = s4_selective_scan_workspace_bytes(a->batch, a->L, a->H, a->N, a->G);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st{nullptr, 0u};
  if (a->ws || need > s4impl::kStatusBytes) {
    const s4_status w = ws_ok(a->ws, a->ws_bytes, need);
    if (w != S4_OK) return w;
    bool chain;
    if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  }
  return cuda_status(s4impl::launch_selective_scan(*a, st, s));
}

size_t s4_selective_scan_bwd_workspace_bytes(int batch, int L, int H, int N, int G) {
  if (!scan_sizes_ok(batch, L, H, N, G)) return 0;
  return s4impl::selective_bwd_bytes(batch, L, H, N, G);
}

s4_status s4_selective_scan_bwd(const s4_selective_bwd_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || !scan_sizes_ok(a->batch, a->L, a->H, a->N, a->G)) return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype);
  if (!rows_ok(a->x, a->dtype) || !rows_ok(a->dt, a->dtype) || (a->z.p && !rows_ok(a->z, a->dtype)) ||
      !rows_ok(a->B, a->dtype) || !rows_ok(a->C, a->dtype) || !rows_ok(a->dy, a->dtype) || !rows_ok(a->dx, a->dtype) ||
      !rows_ok(a->ddt, a->dtype) || (a->z.p && !rows_ok(a->dz, a->dtype)) || (!a->z.p && a->dz.p) || a->B_group < 0 ||
      a->C_group < 0)
    return S4_ERR_INVALID_ARG;
  if (!a->dB || !a->dC || !a->A || !a->dA || !a->D != !a->dD || !a->dt_bias != !a->ddt_bias || !aligned(a->dB, e) ||
      !aligned(a->dC, e) || !aligned(a->A, 4) || !aligned(a->dA, 4) || !aligned(a->D, 4) || !aligned(a->dD, 4) ||
      !aligned(a->dt_bias, 4) || !aligned(a->ddt_bias, 4) || !aligned(a->lengths, 4) || !aligned(a->state0, 4) ||
      !aligned(a->dstate, 4) || !aligned(a->dstate0, 4) || (a->dstate0 && a->dstate0 == a->dstate))
    return S4_ERR_INVALID_ARG;
  const size_t need = s4_selective_scan_bwd_workspace_bytes(a->batch, a->L, a->H, a->N, a->G);
  if (need == 0) return S4_ERR_INVALID_ARG;
  const s4_status w = ws_ok(a->ws, a->ws_bytes, need);
  if (w != S4_OK) return w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st;
  bool chain;
  if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  return cuda_status(s4impl::launch_selective_bwd(*a, st, s));
}

s4_status s4_block_norm_fwd(const s4_block_norm_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || a->rows < 1 || a->rows > INT_MAX || a->H < 1 || a->H > kMaxNormChannels ||
      !(a->eps >= 0.f))
    return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype), er = a->res_f32 ? 4 : e;
  if (!a->o || !a->h_out || !a->y != !a->w_pre || !aligned(a->o, e) || !aligned(a->gate, e) || !aligned(a->h, er) ||
      !aligned(a->h_out, er) || !aligned(a->y, e) || !aligned(a->w_post, 4) || !aligned(a->scale, 4) ||
      !aligned(a->w_pre, 4) || a->o_row < 0 || a->gate_row < 0 || a->h_row < 0 || a->h_out_row < 0 || a->y_row < 0)
    return S4_ERR_INVALID_ARG;
  // in place: each row at its own address (else a row would replace another that is still needed)
  if (a->h_out == a->h && a->rows > 1 && a->h_out_row != a->h_row) return S4_ERR_INVALID_ARG;
  return cuda_status(s4impl::launch_block_norm(*a, static_cast<cudaStream_t>(stream)));
}

size_t s4_block_norm_bwd_workspace_bytes(long long rows, int H) {
  if (rows < 1 || rows > INT_MAX || H < 1 || H > kMaxNormChannels) return 0;
  return s4impl::kStatusBytes + s4impl::align256(s4impl::block_norm_bwd_scratch(rows, H));
}

s4_status s4_block_norm_bwd(const s4_block_norm_bwd_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || a->rows < 1 || a->rows > INT_MAX || a->H < 1 || a->H > kMaxNormChannels ||
      !(a->eps >= 0.f))
    return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype), er = a->res_f32 ? 4 : e;
  if (!a->o || !a->do_ || (!a->dy && !a->dh_out) || (a->dy && !a->w_pre) || !a->gate != !a->dgate || !a->h != !a->dh ||
      !a->w_post != !a->dw_post || !a->scale != !a->dscale || !a->w_pre != !a->dw_pre)
    return S4_ERR_INVALID_ARG;
  if (!aligned(a->o, e) || !aligned(a->gate, e) || !aligned(a->h, er) || !aligned(a->dy, e) ||
      !aligned(a->dh_out, er) || !aligned(a->do_, e) || !aligned(a->dgate, e) || !aligned(a->dh, er) ||
      !aligned(a->w_post, 4) || !aligned(a->scale, 4) || !aligned(a->w_pre, 4) || !aligned(a->dw_post, 4) ||
      !aligned(a->dscale, 4) || !aligned(a->dw_pre, 4))
    return S4_ERR_INVALID_ARG;
  if (a->o_row < 0 || a->gate_row < 0 || a->h_row < 0 || a->dy_row < 0 || a->dh_out_row < 0 || a->do_row < 0 ||
      a->dgate_row < 0 || a->dh_row < 0)
    return S4_ERR_INVALID_ARG;
  const s4_status w = ws_ok(a->ws, a->ws_bytes, s4_block_norm_bwd_workspace_bytes(a->rows, a->H));
  if (w != S4_OK) return w;
  return cuda_status(s4impl::launch_block_norm_bwd(*a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
