// The tile kernel's instances over a cache of 4 bits.

#include "paged_attention.cuh"

namespace nvfp4 {
namespace {
__device__ __forceinline__ int* status_word(const AttnParams& p) { return p.status; }
}  // namespace
}  // namespace nvfp4

nvfp4_status nvfp4::attn::launch_tiles_4bit(const TilePlan& t, const AttnParams& p, int grid, cudaStream_t stream) {
    if (p.D == t.dp) return dispatch_tile<NVFP4_E2M1, false, true>(t, p, grid, stream);
    return dispatch_tile<NVFP4_E2M1, false, false>(t, p, grid, stream);
}
