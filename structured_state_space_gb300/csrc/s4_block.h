// Host-side interfaces of the selective block's operators (short causal
// convolution, selective scan, block norms), beside s4_internal.h.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>

#include "s4.h"
#include "s4_internal.h"

namespace s4impl {

// Device status bit of a length or state slot out of range (the lower bits are
// those of s4_dev.cuh).
constexpr unsigned ST_BAD_INDEX = 64u;

// The status of a call on `s` (defined in s4_api.cu).
bool call_status(void* ws, cudaStream_t s, St* st, bool* chain);

inline int dtype_bytes(int dtype) { return dtype == S4_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) { return dtype == S4_F32 || dtype == S4_BF16 || dtype == S4_F16; }

// Device bytes of the workspace's status block, before its other sections.
constexpr size_t kStatusBytes = 256;
inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }
// Bytes between two sections of a workspace: none, but in the bounds-checked build, where an access
// beyond a section's end is not to land in the next.
#ifdef S4_BOUNDS_CHECK
constexpr size_t kGap = 4096;
#else
constexpr size_t kGap = 0;
#endif

cudaError_t launch_short_conv(const s4_short_conv_args& a, St st, cudaStream_t s);
size_t short_conv_bwd_scratch(int batch, int L, int H, int W);
cudaError_t launch_short_conv_bwd(const s4_short_conv_bwd_args& a, St st, cudaStream_t s);
size_t selective_scratch(int batch, int L, int H, int N, int G);
cudaError_t launch_selective_scan(const s4_selective_args& a, St st, cudaStream_t s);
size_t selective_bwd_bytes(int batch, int L, int H, int N, int G);
cudaError_t launch_selective_bwd(const s4_selective_bwd_args& a, St st, cudaStream_t s);
cudaError_t launch_block_norm(const s4_block_norm_args& a, cudaStream_t s);
size_t block_norm_bwd_scratch(long long rows, int H);
cudaError_t launch_block_norm_bwd(const s4_block_norm_bwd_args& a, cudaStream_t s);

#ifdef S4_BOUNDS_CHECK
unsigned long long oob_short_conv();
unsigned long long oob_selective();
unsigned long long oob_selective_bwd();
unsigned long long oob_block_norm();
#endif

}  // namespace s4impl
