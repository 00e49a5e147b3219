// The tile kernel's instances over a cache of 4 bits.

#include "paged_attention.cuh"

nvfp4_status nvfp4::attn::launch_tiles_4bit(const TilePlan& t, const AttnParams& p, int grid, cudaStream_t stream) {
    if (p.slopes || p.cap > 0.0f) return dispatch_tile<NVFP4_E2M1, true>(t, p, grid, stream);
    return dispatch_tile<NVFP4_E2M1, false>(t, p, grid, stream);
}
