// The tile kernel's instances for capped or biased scores over a cache of 4 bits.

#include "paged_attention.cuh"

namespace nvfp4 {
namespace {
__device__ __forceinline__ int* status_word(const AttnParams& p) { return p.status; }
}  // namespace
}  // namespace nvfp4

nvfp4_status nvfp4::attn::launch_tiles_4bit_scored(const TilePlan& t, const AttnParams& p, int grid, cudaStream_t stream) {
    if (p.D == t.dp) return dispatch_tile<NVFP4_E2M1, true, true>(t, p, grid, stream);
    return dispatch_tile<NVFP4_E2M1, true, false>(t, p, grid, stream);
}
