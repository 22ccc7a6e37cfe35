// The tcgen05 attention kernel's launcher (pa_attn_tc.cu).
#pragma once

#include <cuda_runtime.h>

namespace pa {

struct AttnMaps;
struct CacheAttnParams;

constexpr int kTcMaxWidth = 4096;  // blocks of a request whose rows have lists (the tiles leave no room for more bit sets)

// `grid` CTAs over slices of the items (fmt: 0 FP8, 1 NVFP4); partial results
// as pa_attn_kernel leaves them, one sum of weights a block.
cudaError_t launch_attn_tc(int fmt, const AttnMaps &maps, const CacheAttnParams &a, int grid, bool pdl, cudaStream_t stream);

}  // namespace pa
