// Attention of each sequence's newest tokens over its paged key-value cache.
//
//   s_j = scale * q . k_j  over the keys j that the row sees,   m = max s_j,   l = sum exp(s_j - m)
//   out = sum exp(s_j - m) v_j / l,   lse = m + log l
//
// Keys are taken in one pass: a part of them leaves (m, l, sum exp(s - m) v), and two parts join by
// rescaling both to the larger maximum.

#include "ops_common.cuh"

#include <cmath>

namespace nvfp4 {
namespace {

using namespace ops;

__device__ int g_attention_status;

constexpr int kMaxRows = 8;
constexpr int kMaxDim = 512;

struct AttnParams {
    const __nv_bfloat16* q;
    const void* cache[2];       // k, v
    int64_t page_stride[2];     // elements between pages
    const float* cache_scale[2];
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lengths;
    __nv_bfloat16* out;
    float* lse;
    int64_t q_ts, q_hs;
    int seqs, rows, hq, hk, group, D, pages, max_pages, page, window, fp8;
    float scale;
};

__device__ __forceinline__ int length_of(const AttnParams& p, int b) {
    const int n = p.lengths[b], most = p.max_pages * p.page;
    if (n < 0 || n > most) {
        atomicOr(&g_attention_status, NVFP4_DEV_BAD_PAGE);
        return n < 0 ? 0 : most;
    }
    return n;
}

// Values d, d + 32, ... of a key or value row, one lane each.
template <int V>
__device__ __forceinline__ void load_row(const AttnParams& p, int which, int64_t at, int lane, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = lane + 32 * i;
        v[i] = 0.0f;
        if (d < p.D) {
            if (p.fp8) v[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(
                                   e4m3x2_f16x2(static_cast<const uint8_t*>(p.cache[which])[at + d]) & 0xffffu)));
            else v[i] = load_one(static_cast<const __nv_bfloat16*>(p.cache[which]) + at + d);
        }
    }
}

constexpr int kScalarWarps = 4;

// One CTA per (query row, query head); each warp takes every fourth key. Any head size up to 512,
// any page size, any alignment.
__global__ void __launch_bounds__(kScalarWarps * 32) paged_attention_scalar_kernel(const __grid_constant__ AttnParams p) {
    constexpr int V = kMaxDim / 32;
    __shared__ float part[kScalarWarps][kMaxDim];
    __shared__ float pm[kScalarWarps], pl[kScalarWarps];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y, hk = h / p.group, b = static_cast<int>(t) / p.rows, r = static_cast<int>(t) % p.rows;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = length_of(p, b);
    const int end = n - p.rows + r + 1;
    const int begin = p.window > 0 && end > p.window ? end - p.window : 0;
    float q[V], o[V], m = -INFINITY, l = 0.0f;
    const float ks = p.cache_scale[0] ? p.cache_scale[0][hk] : 1.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < p.D ? load_one(p.q + t * p.q_ts + h * p.q_hs + d) : 0.0f;
        o[i] = 0.0f;
    }
    for (int j = begin + warp; j < end; j += kScalarWarps) {
        const int pi = j / p.page, page = p.table[b * p.table_stride + pi];
        if (page < 0 || page >= p.pages) {
            if (lane == 0) atomicOr(&g_attention_status, NVFP4_DEV_BAD_PAGE);
            continue;
        }
        const int64_t row = (static_cast<int64_t>(hk) * p.page + (j - pi * p.page)) * p.D;
        float x[V], s = 0.0f;
        load_row(p, 0, page * p.page_stride[0] + row, lane, x);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= p.scale * ks;
        load_row(p, 1, page * p.page_stride[1] + row, lane, x);
        if (s == -INFINITY) continue;  // weight zero, also while every score was -inf
        const float top = fmaxf(m, s);
        const float keep = m == -INFINITY ? 0.0f : expf(m - top), add = expf(s - top);
        m = top;
        l = l * keep + add;
#pragma unroll
        for (int i = 0; i < V; ++i) o[i] = fmaf(add, x[i], o[i] * keep);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) part[warp][lane + 32 * i] = o[i];
    if (lane == 0) { pm[warp] = m; pl[warp] = l; }
    __syncthreads();
    float top = -INFINITY, total = 0.0f, w[kScalarWarps];
    for (int i = 0; i < kScalarWarps; ++i) top = fmaxf(top, pm[i]);
    for (int i = 0; i < kScalarWarps; ++i) {
        w[i] = pl[i] == 0.0f ? 0.0f : pm[i] == -INFINITY ? 1.0f : expf(pm[i] - top);  // NaN scores leave m at -inf
        total += pl[i] * w[i];
    }
    const float vs = p.cache_scale[1] ? p.cache_scale[1][hk] : 1.0f;
    for (int d = threadIdx.x; d < p.D; d += blockDim.x) {
        float sum = 0.0f;
        for (int i = 0; i < kScalarWarps; ++i) if (w[i] != 0.0f) sum += part[i][d] * w[i];
        p.out[(t * p.hq + h) * p.D + d] = __float2bfloat16_rn(total == 0.0f ? 0.0f : sum * vs / total);
    }
    if (p.lse && threadIdx.x == 0) p.lse[t * p.hq + h] = total == 0.0f ? -INFINITY : top + logf(total);
}

cudaError_t read_status(int* bits) {
    const int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, g_attention_status, sizeof(int));
    return e != cudaSuccess || *bits == 0 ? e : cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(int));
}
const bool g_registered = register_status(read_status);

bool sizes_ok(int seqs, int rows, int hq, int hk, int dim) {
    return seqs >= 0 && rows >= 0 && rows <= kMaxRows && hq >= 0 && hk >= 0 && dim >= 0 && (hk == 0 ? hq == 0 : hq % hk == 0);
}

}  // namespace
}  // namespace nvfp4

extern "C" int64_t nvfp4_attention_workspace_bytes(int seqs, int rows, int q_heads, int kv_heads, int head_dim) {
    using namespace nvfp4;
    if (!sizes_ok(seqs, rows, q_heads, kv_heads, head_dim) || head_dim > kMaxDim) return -1;
    return 256;
}

extern "C" nvfp4_status nvfp4_paged_attention(const nvfp4_paged_attention_args* a, void* stream) {
    using namespace nvfp4;
    using namespace nvfp4::ops;
    if (!a) return NVFP4_ERR_NULL;
    if (!sizes_ok(a->seqs, a->rows, a->q_heads, a->kv_heads, a->head_dim) || a->pages < 0 || a->max_pages < 0 ||
        a->page_size < 1 || a->window < 0)
        return NVFP4_ERR_SHAPE;
    if (a->cache_type != NVFP4_BF16 && a->cache_type != NVFP4_E4M3) return NVFP4_ERR_DTYPE;
    if (a->seqs == 0 || a->rows == 0 || a->q_heads == 0 || a->head_dim == 0) return NVFP4_OK;
    if (a->head_dim > kMaxDim || a->q_heads > 65535 || static_cast<int64_t>(a->seqs) * a->rows > (1 << 30) ||
        static_cast<int64_t>(a->max_pages) * a->page_size > (1 << 24))
        return NVFP4_ERR_UNSUPPORTED;
    if (!a->q || !a->k_cache || !a->v_cache || !a->page_table || !a->lengths || !a->out || !a->workspace)
        return NVFP4_ERR_NULL;
    if (!aligned(a->workspace, 256)) return NVFP4_ERR_ALIGN;
    if (a->workspace_bytes < nvfp4_attention_workspace_bytes(a->seqs, a->rows, a->q_heads, a->kv_heads, a->head_dim))
        return NVFP4_ERR_SHAPE;
    AttnParams p{};
    p.q = static_cast<const __nv_bfloat16*>(a->q);
    p.cache[0] = a->k_cache; p.cache[1] = a->v_cache;
    p.page_stride[0] = a->k_page_stride; p.page_stride[1] = a->v_page_stride;
    p.cache_scale[0] = a->k_scale; p.cache_scale[1] = a->v_scale;
    p.table = a->page_table; p.table_stride = a->table_stride; p.lengths = a->lengths;
    p.out = static_cast<__nv_bfloat16*>(a->out); p.lse = a->lse;
    p.q_ts = a->q_token_stride; p.q_hs = a->q_head_stride;
    p.seqs = a->seqs; p.rows = a->rows; p.hq = a->q_heads; p.hk = a->kv_heads; p.group = a->q_heads / a->kv_heads;
    p.D = a->head_dim; p.pages = a->pages; p.max_pages = a->max_pages; p.page = a->page_size;
    p.window = a->window; p.fp8 = a->cache_type == NVFP4_E4M3; p.scale = a->scale;
    return launch(paged_attention_scalar_kernel, dim3(a->seqs * a->rows, a->q_heads), dim3(kScalarWarps * 32), 0,
                  static_cast<cudaStream_t>(stream), p);
}
