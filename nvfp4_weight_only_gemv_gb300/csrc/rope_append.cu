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
    int tokens_per_cta, lanes_log2;  // vector kernel
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

// Vector kernel: a lane holds 8 values of a head as two vectors of 4, chosen so that both members of
// each rotated pair are its own: in halves, values 4i.. and half + 4i..; interleaved, or beyond the
// rotary part, 8 neighbours. D / 8 lanes make a head. A CTA takes a few tokens: their cosines and
// sines are formed once, in shared memory, and serve all heads of q and k.
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack4_e4m3(const float (&v)[4]) {
    return pack_e4m3(v[0], v[1]) | pack_e4m3(v[2], v[3]) << 16;
}

template <typename XT>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const __grid_constant__ AppendParams p) {
    extern __shared__ __align__(16) float2 cs[];  // [tokens_per_cta][half]
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.tokens_per_cta;
    const int tokens = min(p.tokens_per_cta, p.T - t0);
    const int heads = p.hq + 2 * p.hk, lanes = 1 << p.lanes_log2;
    const int i = tid & (lanes - 1);        // lane within the head
    const bool live = 8 * i < p.D;
    // offsets of the lane's two vectors, and its first rotated pair (-1: none)
    int oa = 8 * i, ob = 8 * i + 4, pair = -1;
    if (8 * i < 2 * p.half) {
        pair = 4 * i;
        if (!p.interleaved) { oa = 4 * i; ob = p.half + 4 * i; }
    }
    for (int j = tid; j < tokens * p.half; j += kThreads) {
        const int n = p.positions[t0 + j / p.half];
        float2 v = cos_sin(n < 0 ? 0 : n, p.inv_freq[j % p.half]);
        cs[j] = make_float2(v.x * p.mscale, v.y * p.mscale);
    }
    __syncthreads();
    const int step = kThreads >> p.lanes_log2;  // heads at a time
    const int first = blockIdx.y * step + (tid >> p.lanes_log2), stride = gridDim.y * step;
    // every lane of a warp passes through every turn: the norm's shuffles need them all
    const int turns = (tokens * heads - blockIdx.y * step + stride - 1) / stride;
    for (int k = 0, item = first; k < turns; ++k, item += stride) {
        const bool in = item < tokens * heads && live;
        const int tk = in ? item / heads : 0;
        int h = in ? item - tk * heads : 0;
        const int t = t0 + tk;
        const int part = h < p.hq ? 0 : h < p.hq + p.hk ? 1 : 2;
        h -= part == 0 ? 0 : part == 1 ? p.hq : p.hq + p.hk;
        float a[4] = {}, b[4] = {};
        if (in) {
            const XT* x = static_cast<const XT*>(p.x[part]) + t * p.ts[part] + h * p.hs[part];
            load_vec(x + oa, a);
            load_vec(x + ob, b);
        }
        const void* w = part == 0 ? p.q_norm : part == 1 ? p.k_norm : nullptr;
        if (p.q_norm || p.k_norm) {
            float sum = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum = fmaf(a[e], a[e], fmaf(b[e], b[e], sum));
            for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (w && in) {
                const float rstd = rsqrtf(sum / static_cast<float>(p.D) + p.eps);
                float wa[4], wb[4];
                if (p.norm_type == NVFP4_F32) {
                    load_vec(static_cast<const float*>(w) + oa, wa);
                    load_vec(static_cast<const float*>(w) + ob, wb);
                } else {
                    load_vec(static_cast<const __nv_bfloat16*>(w) + oa, wa);
                    load_vec(static_cast<const __nv_bfloat16*>(w) + ob, wb);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) { a[e] *= rstd * wa[e]; b[e] *= rstd * wb[e]; }
            }
        }
        if (!in) continue;
        if (part < 2 && pair >= 0) {
            float2 r[4];
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                const float4 v = *reinterpret_cast<const float4*>(cs + tk * p.half + pair + e);
                r[e] = make_float2(v.x, v.y);
                r[e + 1] = make_float2(v.z, v.w);
            }
            if (p.interleaved) {
                auto turn = [](float& u, float& v, float2 c) {
                    const float x = u * c.x - v * c.y;
                    v = v * c.x + u * c.y;
                    u = x;
                };
                turn(a[0], a[1], r[0]); turn(a[2], a[3], r[1]); turn(b[0], b[1], r[2]); turn(b[2], b[3], r[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float x = a[e] * r[e].x - b[e] * r[e].y;
                    b[e] = b[e] * r[e].x + a[e] * r[e].y;
                    a[e] = x;
                }
            }
        }
        const int n = p.positions[t];
        if (part == 0) {
            if (n < 0) {
#pragma unroll
                for (int e = 0; e < 4; ++e) a[e] = b[e] = 0.0f;
            }
            __nv_bfloat16* to = p.q_out + (static_cast<int64_t>(t) * p.hq + h) * p.D;
            store_vec(to + oa, a);
            store_vec(to + ob, b);
            continue;
        }
        Place at;
        if (!place_of(p, t, n, at)) continue;
        const int64_t to = at.page * p.page_stride[part - 1] + (static_cast<int64_t>(h) * p.page + at.slot) * p.D;
        if (p.fp8) {
            const float* sc = p.cache_scale[part - 1];
            const float s = sc ? sc[h] : 1.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) { a[e] /= s; b[e] /= s; }
            uint8_t* c = static_cast<uint8_t*>(p.cache[part - 1]) + to;
            *reinterpret_cast<uint32_t*>(c + oa) = pack4_e4m3(a);
            *reinterpret_cast<uint32_t*>(c + ob) = pack4_e4m3(b);
        } else {
            __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.cache[part - 1]) + to;
            store_vec(c + oa, a);
            store_vec(c + ob, b);
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
    // Vectors of 4 values: 8-byte pieces of bf16, 16-byte pieces of fp32, 4-byte pieces of codes.
    const int xb = a->x_type == NVFP4_F32 ? 16 : 8, nb = p.norm_type == NVFP4_F32 ? 16 : 8;
    const int cb = p.fp8 ? 4 : 8;
    bool vec = p.D % 8 == 0 && p.D <= 256 && p.half % 4 == 0 && aligned(p.q_out, 8) && aligned(p.q_norm, nb) &&
               aligned(p.k_norm, nb);
    for (int i = 0; i < 3; ++i) vec = vec && aligned(p.x[i], xb) && p.ts[i] % 4 == 0 && p.hs[i] % 4 == 0;
    for (int i = 0; i < 2; ++i) vec = vec && aligned(p.cache[i], cb) && p.page_stride[i] % 4 == 0;
    if (vec && host_variant() != 1) {
        while ((8 << p.lanes_log2) < p.D) ++p.lanes_log2;
        const int step = kThreads >> p.lanes_log2, heads = p.hq + 2 * p.hk, sms = host_sm_count();
        // Few tokens: one a CTA, its heads over several CTAs. Many: 4 a CTA share one barrier.
        p.tokens_per_cta = p.T >= 8 * sms ? 4 : 1;
        const int groups = (p.T + p.tokens_per_cta - 1) / p.tokens_per_cta;
        int parts = p.T >= 2 * sms ? 1 : (heads + step - 1) / step;
        const dim3 grid(groups, parts);
        const size_t smem = static_cast<size_t>(p.tokens_per_cta) * p.half * sizeof(float2);
        return a->x_type == NVFP4_F32 ? launch(rope_append_kernel<float>, grid, dim3(kThreads), smem, st, p)
                                      : launch(rope_append_kernel<__nv_bfloat16>, grid, dim3(kThreads), smem, st, p);
    }
    const dim3 grid(p.T, p.hq + 2 * p.hk);
    return a->x_type == NVFP4_F32 ? launch(rope_append_scalar_kernel<float>, grid, dim3(128), p.D * 4, st, p)
                                  : launch(rope_append_scalar_kernel<__nv_bfloat16>, grid, dim3(128), p.D * 4, st, p);
}
