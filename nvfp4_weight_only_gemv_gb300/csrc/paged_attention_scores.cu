// The tile kernel's instances for capped or biased scores over caches of bf16 and E4M3.

#include "paged_attention.cuh"

namespace nvfp4 {
namespace {
__device__ __forceinline__ int* status_word(const AttnParams& p) { return p.status; }
}  // namespace
}  // namespace nvfp4

nvfp4_status nvfp4::attn::launch_tiles_scored(const TilePlan& t, const AttnParams& p, int grid, cudaStream_t stream) {
    if (p.cache_type == NVFP4_E4M3) return dispatch_tile<NVFP4_E4M3, true>(t, p, grid, stream);
    return dispatch_tile<NVFP4_BF16, true>(t, p, grid, stream);
}
