// Rotary positions of q and k, and the append of k and v to a paged cache.
//
// For token t at position n = positions[t], per head of q and k (v is only appended):
//   u      = x / sqrt(mean(x^2) + eps) * w            (per-head norm; left out without weights)
//   y[a_i] = u[a_i] c_i - u[b_i] s_i,  y[b_i] = u[b_i] c_i + u[a_i] s_i,   i < half
//   c_i, s_i = mscale * cos, sin(n * inv_freq[i])
//   (a_i, b_i) = (i, i + half) or, interleaved, (2i, 2i + 1); the head's other values pass through
// q goes to q_out in bf16, k and v to row n % page of page table[seq][n / page] of the cache
// [pages, kv heads, page, D], in bf16 or as E4M3(value / scale[kv head]).
//
// The kernel moves each value once and is bound by that traffic for prompts, by latency for
// single tokens.

#include "ops_common.cuh"

namespace nvfp4 {
namespace {

using namespace ops;

__device__ int g_append_status;

struct AppendParams {
    const void* x[3];        // q, k, v
    int64_t ts[3], hs[3];    // token and head strides, elements
    const int32_t* positions;
    const int32_t* seq_ids;  // NULL: token t belongs to sequence t / per_seq
    const float* inv_freq;
    const void* q_norm;
    const void* k_norm;
    __nv_bfloat16* q_out;
    void* cache[2];          // k, v
    int64_t page_stride[2];  // elements between pages
    const float* cache_scale[2];
    const int32_t* table;
    int64_t table_stride;
    int T, hq, hk, D, half, seqs, per_seq, pages, max_pages, page;
    int norm_type, interleaved, fp8;
    float mscale, eps;
};

// cos and sin of n * f for a whole n below 2^24. The product is taken exactly as p + e, and whole
// turns are removed in three parts of 2 pi (Cody and Waite, "Software Manual for the Elementary
// Functions", 1980), so the angle keeps its absolute error of about 2^-23 at every position; the
// product alone, rounded to fp32, would be off by up to half a unit in its last place, 0.03 at
// n f = 10^6.
__device__ __forceinline__ float2 cos_sin(int n, float f) {
    const float nf = static_cast<float>(n);
    const float p = nf * f, e = fmaf(nf, f, -p);
    const float k = rintf(p * 0.15915494f);
    float r = fmaf(-k, 0x1.921fb6p+2f, p);
    r = fmaf(-k, -0x1.777a5cp-23f, r);
    r = fmaf(-k, -0x1.ee59dap-48f, r);
    float s, c;
    sincosf(r + e, &s, &c);
    return make_float2(c, s);
}

// Where token t's key and value rows go; false (and a status bit where the position is not
// negative) when there is no such place.
struct Place {
    int64_t page;
    int slot;
};
__device__ __forceinline__ bool place_of(const AppendParams& p, int t, int n, Place& at) {
    if (n < 0) return false;  // a padding token
    const int seq = p.seq_ids ? p.seq_ids[t] : t / p.per_seq;
    const int pi = n / p.page;
    if (seq >= 0 && seq < p.seqs && pi < p.max_pages) {
        const int page = p.table[seq * p.table_stride + pi];
        if (page >= 0 && page < p.pages) {
            at.page = page;
            at.slot = n - pi * p.page;
            return true;
        }
    }
    atomicOr(&g_append_status, NVFP4_DEV_BAD_PAGE);
    return false;
}

// One value a thread, one CTA per (head, token): any head size, alignment and rotary size.
template <typename XT>
__global__ void __launch_bounds__(128) rope_append_scalar_kernel(const __grid_constant__ AppendParams p) {
    extern __shared__ float u[];
    __shared__ float red[4];
    pdl_launch_dependents();
    pdl_wait();
    const int t = blockIdx.x, tid = threadIdx.x;
    int h = blockIdx.y;
    const int part = h < p.hq ? 0 : h < p.hq + p.hk ? 1 : 2;
    h -= part == 0 ? 0 : part == 1 ? p.hq : p.hq + p.hk;
    const int n = p.positions[t];
    const XT* x = static_cast<const XT*>(p.x[part]) + t * p.ts[part] + h * p.hs[part];
    const void* w = part == 0 ? p.q_norm : part == 1 ? p.k_norm : nullptr;
    float sum = 0.0f;
    for (int d = tid; d < p.D; d += 128) {
        const float v = load_one(x + d);
        u[d] = v;
        sum = fmaf(v, v, sum);
    }
    if (w) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if ((tid & 31) == 0) red[tid >> 5] = sum;
        __syncthreads();
        const float rstd = rsqrtf((red[0] + red[1] + red[2] + red[3]) / static_cast<float>(p.D) + p.eps);
        for (int d = tid; d < p.D; d += 128)
            u[d] *= rstd * (p.norm_type == NVFP4_F32 ? static_cast<const float*>(w)[d]
                                                     : load_one(static_cast<const __nv_bfloat16*>(w) + d));
    }
    __syncthreads();
    Place at{0, 0};
    const bool ok = part == 0 ? n >= 0 : place_of(p, t, n, at);
    if (part != 0 && !ok) return;
    for (int d = tid; d < p.D; d += 128) {
        float y = u[d];
        if (part < 2 && d < 2 * p.half) {
            const int i = p.interleaved ? d >> 1 : d % p.half;
            const bool first = p.interleaved ? (d & 1) == 0 : d < p.half;
            const float other = u[p.interleaved ? d ^ 1 : first ? d + p.half : d - p.half];
            float2 cs = cos_sin(n < 0 ? 0 : n, p.inv_freq[i]);
            cs.x *= p.mscale;
            cs.y *= p.mscale;
            y = first ? y * cs.x - other * cs.y : y * cs.x + other * cs.y;
        }
        if (part == 0) {
            p.q_out[(static_cast<int64_t>(t) * p.hq + h) * p.D + d] = __float2bfloat16_rn(ok ? y : 0.0f);
        } else {
            const int64_t to = at.page * p.page_stride[part - 1] + (static_cast<int64_t>(h) * p.page + at.slot) * p.D + d;
            if (p.fp8) {
                const float* sc = p.cache_scale[part - 1];
                static_cast<uint8_t*>(p.cache[part - 1])[to] = static_cast<uint8_t>(pack_e4m3(y / (sc ? sc[h] : 1.0f), 0.0f));
            } else {
                static_cast<__nv_bfloat16*>(p.cache[part - 1])[to] = __float2bfloat16_rn(y);
            }
        }
    }
}

cudaError_t read_status(int* bits) {
    const int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, g_append_status, sizeof(int));
    return e != cudaSuccess || *bits == 0 ? e : cudaMemcpyToSymbol(g_append_status, &zero, sizeof(int));
}
const bool g_registered = register_status(read_status);

}  // namespace
}  // namespace nvfp4

extern "C" nvfp4_status nvfp4_rope_append(const nvfp4_rope_append_args* a, void* stream) {
    using namespace nvfp4;
    using namespace nvfp4::ops;
    if (!a) return NVFP4_ERR_NULL;
    const int hq = a->q ? a->q_heads : 0;
    if (a->tokens < 0 || hq < 0 || a->kv_heads < 0 || a->head_dim < 0 || a->rotary_half < 0 || a->seqs < 0 ||
        a->pages < 0 || a->max_pages < 0 || a->page_size < 1 || 2 * static_cast<int64_t>(a->rotary_half) > a->head_dim ||
        !(a->eps >= 0.0f))
        return NVFP4_ERR_SHAPE;
    if ((a->x_type != NVFP4_F32 && a->x_type != NVFP4_BF16) || (a->cache_type != NVFP4_BF16 && a->cache_type != NVFP4_E4M3) ||
        ((a->q_norm || a->k_norm) && a->norm_type != NVFP4_F32 && a->norm_type != NVFP4_BF16))
        return NVFP4_ERR_DTYPE;
    if (a->tokens == 0 || a->head_dim == 0 || hq + a->kv_heads == 0) return NVFP4_OK;
    if (a->head_dim > 1024 || static_cast<int64_t>(hq) + 2 * static_cast<int64_t>(a->kv_heads) > 65535 ||
        static_cast<int64_t>(a->max_pages) * a->page_size > (1 << 24))
        return NVFP4_ERR_UNSUPPORTED;
    if (!a->positions || (a->rotary_half && !a->inv_freq) || (hq && !a->q_out) ||
        (a->kv_heads && (!a->k || !a->v || !a->k_cache || !a->v_cache || !a->page_table)))
        return NVFP4_ERR_NULL;
    if (a->kv_heads && (a->seqs == 0 || (!a->seq_ids && a->tokens % a->seqs))) return NVFP4_ERR_SHAPE;
    AppendParams p{};
    p.x[0] = a->q; p.x[1] = a->k; p.x[2] = a->v;
    p.ts[0] = a->q_token_stride; p.ts[1] = a->k_token_stride; p.ts[2] = a->v_token_stride;
    p.hs[0] = a->q_head_stride; p.hs[1] = a->k_head_stride; p.hs[2] = a->v_head_stride;
    p.positions = a->positions; p.seq_ids = a->seq_ids; p.inv_freq = a->inv_freq;
    p.q_norm = a->q_norm; p.k_norm = a->k_norm;
    p.q_out = static_cast<__nv_bfloat16*>(a->q_out);
    p.cache[0] = a->k_cache; p.cache[1] = a->v_cache;
    p.page_stride[0] = a->k_page_stride; p.page_stride[1] = a->v_page_stride;
    p.cache_scale[0] = a->k_scale; p.cache_scale[1] = a->v_scale;
    p.table = a->page_table; p.table_stride = a->table_stride;
    p.T = a->tokens; p.hq = hq; p.hk = a->kv_heads; p.D = a->head_dim; p.half = a->rotary_half;
    p.seqs = a->seqs; p.per_seq = a->seqs > 0 ? (a->tokens + a->seqs - 1) / a->seqs : 1;
    p.pages = a->pages; p.max_pages = a->max_pages; p.page = a->page_size;
    p.norm_type = a->norm_type; p.interleaved = a->interleaved; p.fp8 = a->cache_type == NVFP4_E4M3;
    p.mscale = a->mscale; p.eps = a->eps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(p.T, p.hq + 2 * p.hk);
    return a->x_type == NVFP4_F32 ? launch(rope_append_scalar_kernel<float>, grid, dim3(128), p.D * 4, st, p)
                                  : launch(rope_append_scalar_kernel<__nv_bfloat16>, grid, dim3(128), p.D * 4, st, p);
}
