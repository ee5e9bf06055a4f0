// C ABI of linear attention, rotary positions, layer norm and the vocabulary loss (declared in
// include/s4.h): argument checks on the host, then the launches on the caller's stream.
#include <limits.h>
#include <stdint.h>

#include <cmath>

#include "s4.h"
#include "s4_sequence.h"

namespace {

constexpr int kMaxBatch = 65535;
constexpr int kMaxLen = 1 << 24;
constexpr int kMaxHeads = 4096;
constexpr int kMaxWidth = 256;
constexpr int kMaxChannels = 16384;
constexpr long long kMaxRows = 1 << 22;

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
// A strided array of heads: present, aligned to its elements, strides not negative.
template <typename Heads>
bool heads_ok(const Heads& r, int dtype) {
  return r.p && aligned(r.p, s4impl::dtype_bytes(dtype)) && r.batch >= 0 && r.row >= 0 && r.head >= 0;
}
// The same of an output, whose elements lie apart: no stride of 0 in a dimension of more than one.
bool out_ok(const s4_heads_out& r, int dtype, int batch, int L, int heads) {
  return heads_ok(r, dtype) && (batch == 1 || r.batch > 0) && (L == 1 || r.row > 0) && (heads == 1 || r.head > 0);
}
bool tokens_ok(int batch, int L, int H, int G) {
  return batch >= 1 && batch <= kMaxBatch && L >= 1 && L <= kMaxLen && H >= 1 && H <= kMaxHeads && G >= 1 && G <= H;
}
bool attention_ok(int batch, int L, int H, int G, int K, int V) {
  return tokens_ok(batch, L, H, G) && H % G == 0 && K >= 1 && K <= kMaxWidth && V >= 1 && V <= kMaxWidth;
}
s4_status ws_ok(const void* ws, size_t bytes, size_t need) {
  return ws != nullptr && aligned(ws, 256) && bytes >= need ? S4_OK : S4_ERR_WORKSPACE;
}
s4_status cuda_status(cudaError_t e) { return e == cudaSuccess ? S4_OK : S4_ERR_CUDA; }

// What both directions of the vocabulary loss take.
template <typename Args>
bool loss_ok(const Args* a) {
  if (!a || !s4impl::dtype_ok(a->dtype) || a->rows < 1 || a->rows > kMaxRows || a->H < 1 || a->H > kMaxChannels ||
      a->V < 1 || a->V > kMaxRows)
    return false;
  const int e = s4impl::dtype_bytes(a->dtype);
  return a->h && a->w && a->targets && aligned(a->h, e) && aligned(a->w, e) && aligned(a->targets, a->wide_targets ? 8 : 4) &&
         a->h_row >= 0 && a->w_row >= 0;
}

}  // namespace

extern "C" {

size_t s4_linear_attention_workspace_bytes(int batch, int L, int H, int G, int K, int V) {
  if (!attention_ok(batch, L, H, G, K, V)) return 0;
  return s4impl::kStatusBytes + s4impl::linear_attention_scratch(batch, L, H, K, V);
}

s4_status s4_linear_attention_fwd(const s4_linear_attention_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || !attention_ok(a->batch, a->L, a->H, a->G, a->K, a->V)) return S4_ERR_INVALID_ARG;
  if (!heads_ok(a->q, a->dtype) || !heads_ok(a->k, a->dtype) || !heads_ok(a->v, a->dtype) ||
      !out_ok(a->o, a->dtype, a->batch, a->L, a->H) || a->o.p == a->q.p || a->o.p == a->k.p || a->o.p == a->v.p ||
      !a->log_decay || !aligned(a->log_decay, 4) || !aligned(a->lengths, 4) || !aligned(a->index, 4) || !aligned(a->state, 4) ||
      !aligned(a->state_out, 4))
    return S4_ERR_INVALID_ARG;
  if ((a->state || a->state_out) && (a->slots < 1 || (!a->index && a->slots < a->batch))) return S4_ERR_INVALID_ARG;
  const size_t need = s4_linear_attention_workspace_bytes(a->batch, a->L, a->H, a->G, a->K, a->V);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st{nullptr, 0u};
  if (a->ws || need > s4impl::kStatusBytes) {
    const s4_status w = ws_ok(a->ws, a->ws_bytes, need);
    if (w != S4_OK) return w;
    bool chain;
    if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  }
  return cuda_status(s4impl::launch_linear_attention(*a, st, s));
}

size_t s4_linear_attention_bwd_workspace_bytes(int batch, int L, int H, int G, int K, int V) {
  if (!attention_ok(batch, L, H, G, K, V)) return 0;
  return s4impl::kStatusBytes + s4impl::linear_attention_bwd_scratch(batch, L, H, G, K, V);
}

s4_status s4_linear_attention_bwd(const s4_linear_attention_bwd_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || !attention_ok(a->batch, a->L, a->H, a->G, a->K, a->V) ||
      !std::isfinite(a->scale) || !std::isfinite(1.f / a->scale))
    return S4_ERR_INVALID_ARG;
  const s4_heads* in[] = {&a->q, &a->k, &a->v, &a->dout};
  const s4_heads_out* out[] = {&a->dq, &a->dk, &a->dv};
  for (const s4_heads* r : in)
    if (!heads_ok(*r, a->dtype)) return S4_ERR_INVALID_ARG;
  for (const s4_heads_out* r : out) {
    if (!out_ok(*r, a->dtype, a->batch, a->L, r == &a->dq ? a->H : a->G)) return S4_ERR_INVALID_ARG;
    for (const s4_heads* i : in)
      if (i->p == r->p) return S4_ERR_INVALID_ARG;
  }
  if (!a->log_decay || !aligned(a->log_decay, 4) || !aligned(a->lengths, 4) || !aligned(a->state0, 4) ||
      !aligned(a->dstate, 4) || !aligned(a->dstate0, 4) || (a->dstate0 && (a->dstate0 == a->dstate || a->dstate0 == a->state0)))
    return S4_ERR_INVALID_ARG;
  const s4_status w =
      ws_ok(a->ws, a->ws_bytes, s4_linear_attention_bwd_workspace_bytes(a->batch, a->L, a->H, a->G, a->K, a->V));
  if (w != S4_OK) return w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st;
  bool chain;
  if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  return cuda_status(s4impl::launch_linear_attention_bwd(*a, st, s));
}

s4_status s4_rotary(const s4_rotary_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || !tokens_ok(a->batch, a->L, a->H, 1) || a->D < 1 || a->D > kMaxWidth || a->R < 1 ||
      2 * a->R > a->D || (a->k.p ? a->G < 1 || a->G > kMaxHeads : a->G != 0) || !a->freqs || !aligned(a->freqs, 8) ||
      !aligned(a->positions, 4) || a->positions_batch < 0)
    return S4_ERR_INVALID_ARG;
  if (!heads_ok(a->q, a->dtype) || !out_ok(a->q_out, a->dtype, a->batch, a->L, a->H) || !a->k.p != !a->k_out.p ||
      (a->k.p && (!heads_ok(a->k, a->dtype) || !out_ok(a->k_out, a->dtype, a->batch, a->L, a->G))))
    return S4_ERR_INVALID_ARG;
  // in place: each head at its own address (else one would replace another that is still needed)
  const auto in_place_ok = [&](const s4_heads& i, const s4_heads_out& o, int heads) {
    return o.p != i.p || ((a->batch == 1 || o.batch == i.batch) && (a->L == 1 || o.row == i.row) && (heads == 1 || o.head == i.head));
  };
  if (!in_place_ok(a->q, a->q_out, a->H) || (a->k.p && (!in_place_ok(a->k, a->k_out, a->G) || a->k_out.p == a->q.p ||
                                                        a->q_out.p == a->k.p || a->k_out.p == a->q_out.p)))
    return S4_ERR_INVALID_ARG;
  return cuda_status(s4impl::launch_rotary(*a, static_cast<cudaStream_t>(stream)));
}

s4_status s4_layer_norm_fwd(const s4_layer_norm_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || a->rows < 1 || a->rows > INT_MAX || a->H < 1 || a->H > kMaxChannels ||
      !(a->eps >= 0.f))
    return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype);
  if (!a->x || !a->y || !aligned(a->x, e) || !aligned(a->y, e) || !aligned(a->w, 4) || !aligned(a->b, 4) || a->x_row < 0 ||
      a->y_row < 0 || (a->rows > 1 && (a->y_row == 0 || (a->y == a->x && a->y_row != a->x_row))))
    return S4_ERR_INVALID_ARG;
  return cuda_status(s4impl::launch_layer_norm(*a, static_cast<cudaStream_t>(stream)));
}

size_t s4_layer_norm_bwd_workspace_bytes(long long rows, int H) {
  if (rows < 1 || rows > INT_MAX || H < 1 || H > kMaxChannels) return 0;
  return s4impl::kStatusBytes + s4impl::align256(s4impl::layer_norm_bwd_scratch(rows, H));
}

s4_status s4_layer_norm_bwd(const s4_layer_norm_bwd_args* a, void* stream) {
  if (!a || !s4impl::dtype_ok(a->dtype) || a->rows < 1 || a->rows > INT_MAX || a->H < 1 || a->H > kMaxChannels ||
      !(a->eps >= 0.f))
    return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype);
  if (!a->x || !a->dy || !a->dx || !aligned(a->x, e) || !aligned(a->dy, e) || !aligned(a->dx, e) || !aligned(a->w, 4) ||
      !aligned(a->dw, 4) || !aligned(a->db, 4) || a->x_row < 0 || a->dy_row < 0 || a->dx_row < 0 || a->dx == a->x ||
      a->dx == a->dy || (a->rows > 1 && a->dx_row == 0))
    return S4_ERR_INVALID_ARG;
  const s4_status w = ws_ok(a->ws, a->ws_bytes, s4_layer_norm_bwd_workspace_bytes(a->rows, a->H));
  if (w != S4_OK) return w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st;  // nothing goes wrong there, but the status in ws is to be this call's
  bool chain;
  if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  return cuda_status(s4impl::launch_layer_norm_bwd(*a, st, s));
}

size_t s4_vocab_loss_workspace_bytes(const s4_vocab_loss_args* a) {
  return loss_ok(a) ? s4impl::kStatusBytes + s4impl::vocab_loss_scratch(*a) : 0;
}

s4_status s4_vocab_loss_fwd(const s4_vocab_loss_args* a, void* stream) {
  if (!loss_ok(a) || !a->loss || !a->lse || !aligned(a->loss, 4) || !aligned(a->lse, 4) || a->loss == a->lse)
    return S4_ERR_INVALID_ARG;
  const s4_status w = ws_ok(a->ws, a->ws_bytes, s4_vocab_loss_workspace_bytes(a));
  if (w != S4_OK) return w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st;
  bool chain;
  if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  return cuda_status(s4impl::launch_vocab_loss(*a, st, s));
}

size_t s4_vocab_loss_bwd_workspace_bytes(const s4_vocab_loss_bwd_args* a) {
  return loss_ok(a) ? s4impl::kStatusBytes + s4impl::vocab_loss_bwd_scratch(*a) : 0;
}

s4_status s4_vocab_loss_bwd(const s4_vocab_loss_bwd_args* a, void* stream) {
  if (!loss_ok(a) || !a->lse || !a->dloss || !a->dh || !a->dw || !aligned(a->lse, 4) || !aligned(a->dloss, 4))
    return S4_ERR_INVALID_ARG;
  const int e = s4impl::dtype_bytes(a->dtype);
  if (!aligned(a->dh, e) || !aligned(a->dw, e) || a->dh == a->h || a->dh == a->w || a->dw == a->h || a->dw == a->w ||
      a->dh == a->dw)
    return S4_ERR_INVALID_ARG;
  const s4_status w = ws_ok(a->ws, a->ws_bytes, s4_vocab_loss_bwd_workspace_bytes(a));
  if (w != S4_OK) return w;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  s4impl::St st;
  bool chain;
  if (!s4impl::call_status(a->ws, s, &st, &chain)) return S4_ERR_CUDA;
  return cuda_status(s4impl::launch_vocab_loss_bwd(*a, st, s));
}

}  // extern "C"
