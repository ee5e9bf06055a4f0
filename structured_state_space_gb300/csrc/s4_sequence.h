// Host-side interfaces of linear attention, rotary positions, layer norm and the vocabulary
// loss, beside s4_block.h.
#pragma once
#include "s4_block.h"

namespace s4impl {

// A workspace's section of so many bytes, with what keeps it from the next.
inline size_t section(size_t bytes) { return bytes ? align256(bytes) + kGap : 0; }

size_t linear_attention_scratch(int batch, int L, int H, int K, int V);
cudaError_t launch_linear_attention(const s4_linear_attention_args& a, St st, cudaStream_t s);
size_t linear_attention_bwd_scratch(int batch, int L, int H, int G, int K, int V);
cudaError_t launch_linear_attention_bwd(const s4_linear_attention_bwd_args& a, St st, cudaStream_t s);
cudaError_t launch_rotary(const s4_rotary_args& a, cudaStream_t s);
cudaError_t launch_layer_norm(const s4_layer_norm_args& a, cudaStream_t s);
size_t layer_norm_bwd_scratch(long long rows, int H);
cudaError_t launch_layer_norm_bwd(const s4_layer_norm_bwd_args& a, St st, cudaStream_t s);
size_t vocab_loss_scratch(const s4_vocab_loss_args& a);
cudaError_t launch_vocab_loss(const s4_vocab_loss_args& a, St st, cudaStream_t s);
size_t vocab_loss_bwd_scratch(const s4_vocab_loss_bwd_args& a);
cudaError_t launch_vocab_loss_bwd(const s4_vocab_loss_bwd_args& a, St st, cudaStream_t s);

#ifdef S4_BOUNDS_CHECK
unsigned long long oob_linear_attention();
unsigned long long oob_linear_attention_tiles();
unsigned long long oob_rotary();
unsigned long long oob_layer_norm();
unsigned long long oob_vocab_loss();
#endif

}  // namespace s4impl
