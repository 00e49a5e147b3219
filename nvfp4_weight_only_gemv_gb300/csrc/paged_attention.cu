// Attention of each sequence's newest tokens over its paged key-value cache: the entry points, the kernel for any
// shape, and the tile kernel's instances for plain scores over caches of bf16 and E4M3.

#include "paged_attention.cuh"

namespace nvfp4 {
namespace {

// A word of this unit's own: by a pointer among their arguments the instances for E4M3, which are short of registers, took 1 to
// 3 % longer (64 x 8191 keys, 16 rows: 174.9 us and 178.9).
__device__ int g_plain_status;
__device__ __forceinline__ int* status_word(const AttnParams&) { return &g_plain_status; }

constexpr int kScalarWarps = 4;

// Values d, d + 32, ... of the key or value at `slot` of a page, one lane each.
template <int V>
__device__ __forceinline__ void load_row(const AttnParams& p, int which, int64_t page, int head, int slot, int lane, float (&v)[V]) {
    if (p.cache_type == NVFP4_E2M1) {
        const int64_t record = static_cast<int64_t>(head) * (p.page / kRecordKeys) + slot / kRecordKeys;
        const uint8_t* const rec = static_cast<const uint8_t*>(p.cache[which]) + page * p.page_stride[which] + record * record_bytes(p.D);
        const int key = slot % kRecordKeys;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int d = lane + 32 * i;
            v[i] = 0.0f;
            if (d < p.D) {
                uint32_t h[4];
                e2m1x8_f16x2(rec[key * (p.D / 2) + d / 2], h);
                v[i] = __half2float(__ushort_as_half(static_cast<unsigned short>(d & 1 ? h[0] >> 16 : h[0] & 0xffffu))) *
                       e4m3_value(rec[8 * p.D + d / 16 * kRecordKeys + key]);
            }
        }
        return;
    }
    const int64_t at = page * p.page_stride[which] + (static_cast<int64_t>(head) * p.page + slot) * p.D;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = lane + 32 * i;
        v[i] = 0.0f;
        if (d < p.D) {
            if (p.cache_type == NVFP4_E4M3) v[i] = e4m3_value(static_cast<const uint8_t*>(p.cache[which])[at + d]);
            else v[i] = load_one(static_cast<const __nv_bfloat16*>(p.cache[which]) + at + d);
        }
    }
}

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
    const float slope = p.slopes ? p.slopes[h] : 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < p.D ? load_one(p.q + t * p.q_ts + h * p.q_hs + d) : 0.0f;
        o[i] = 0.0f;
    }
    for (int j = begin + warp; j < end; j += kScalarWarps) {
        const int pi = j / p.page, page = p.table[b * p.table_stride + pi];
        if (page < 0 || page >= p.pages) {
            if (lane == 0) atomicOr(status_word(p), NVFP4_DEV_BAD_PAGE);
            continue;
        }
        const int slot = j - pi * p.page;
        float x[V], s = 0.0f;
        load_row(p, 0, page, hk, slot, lane, x);
#pragma unroll
        for (int i = 0; i < V; ++i) s = fmaf(q[i], x[i], s);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= p.scale * ks;
        if (p.cap > 0.0f) s = p.cap * tanhf(s / p.cap);
        if (p.slopes) s = fmaf(slope, static_cast<float>(j - (end - 1)), s);
        load_row(p, 1, page, hk, slot, lane, x);
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

bool plan_tile(int dim, int rows, TilePlan* out) {
    TilePlan t;
    if (dim > 256 || rows < 1) return false;
    t.dp = dim <= 64 ? 64 : dim <= 128 ? 128 : 256;
    t.warps = t.dp == 256 ? 8 : 4;
    const int most = 8 * (t.dp == 256 ? 1 : 4) * t.warps;  // rows of a CTA
    t.chunks = (rows + most - 1) / most;
    t.chunk_rows = (rows + t.chunks - 1) / t.chunks;
    t.nt = t.dp == 256 || t.chunk_rows <= 8 ? 1 : t.chunk_rows <= 16 ? 2 : 4;
    while (8 * t.nt * t.row_blocks < t.chunk_rows) t.row_blocks *= 2;
    t.ctas_per_sm = t.dp == 256 ? 1 : t.nt * t.dp <= 128 ? kCtasPerSm : 2;
    *out = t;
    return true;
}

int64_t align256(int64_t v) { return (v + 255) / 256 * 256; }

struct Workspace {
    int64_t part_o, part_ml, bytes;
};
Workspace workspace_of(const TilePlan& t, int sms, int dim) {
    Workspace w;
    const int grid = t.ctas_per_sm * sms;
    w.part_o = align256(4ll * kCtasPerSm * sms * 4);
    w.part_ml = w.part_o + align256(2ll * grid * t.chunk_rows * dim * 4);
    w.bytes = w.part_ml + align256(2ll * grid * t.chunk_rows * 8);
    return w;
}

int sm_count() {
    const int n = host_sm_count();
    return n > 0 ? n : 152;  // sizes asked for without a device: GB300's
}

bool sizes_ok(int seqs, int rows, int hq, int hk, int dim) {
    return seqs >= 0 && rows >= 0 && rows <= kMaxRows && hq >= 0 && hk >= 0 && dim >= 0 && (hk == 0 ? hq == 0 : hq % hk == 0);
}

cudaError_t read_status(int* bits) {
    const int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, g_plain_status, sizeof(int));
    return e != cudaSuccess || *bits == 0 ? e : cudaMemcpyToSymbol(g_plain_status, &zero, sizeof(int));
}
const bool g_status_set = set_attention_status(read_status);

}  // namespace
}  // namespace nvfp4

extern "C" int64_t nvfp4_attention_workspace_bytes(int seqs, int rows, int q_heads, int kv_heads, int head_dim) {
    using namespace nvfp4;
    if (!sizes_ok(seqs, rows, q_heads, kv_heads, head_dim) || head_dim > kMaxDim) return -1;
    TilePlan t;
    const int rows_all = kv_heads ? rows * (q_heads / kv_heads) : 0;
    if (!plan_tile(head_dim, rows_all, &t)) return 256;  // one CTA per row and head: nothing to join
    return workspace_of(t, sm_count(), head_dim).bytes;
}

extern "C" nvfp4_status nvfp4_paged_attention(const nvfp4_paged_attention_args* a, void* stream) {
    return nvfp4_paged_attention_scored(a, nullptr, stream);
}

extern "C" nvfp4_status nvfp4_paged_attention_scored(const nvfp4_paged_attention_args* a, const nvfp4_attention_scores* sc,
                                                     void* stream) {
    using namespace nvfp4;
    using namespace nvfp4::ops;
    if (!a) return NVFP4_ERR_NULL;
    if (!sizes_ok(a->seqs, a->rows, a->q_heads, a->kv_heads, a->head_dim) || a->pages < 0 || a->max_pages < 0 ||
        a->page_size < 1 || a->window < 0)
        return NVFP4_ERR_SHAPE;
    if (sc && sc->softcap != 0.0f && !(sc->softcap >= 0x1p-40f && sc->softcap <= 0x1p40f)) return NVFP4_ERR_SHAPE;
    if ((a->cache_type != NVFP4_BF16 && a->cache_type != NVFP4_E4M3 && a->cache_type != NVFP4_E2M1) ||
        (a->cache_type == NVFP4_BF16 && (a->k_scale || a->v_scale)))
        return NVFP4_ERR_DTYPE;
    if (a->cache_type == NVFP4_E2M1 && (a->head_dim % 16 || a->page_size % kRecordKeys)) return NVFP4_ERR_SHAPE;
    if (a->seqs == 0 || a->rows == 0 || a->q_heads == 0 || a->head_dim == 0) return NVFP4_OK;
    if (a->head_dim > kMaxDim || a->q_heads > 65535 || static_cast<int64_t>(a->seqs) * a->rows > (1 << 30) ||
        static_cast<int64_t>(a->max_pages) * a->page_size > (1 << 24))
        return NVFP4_ERR_UNSUPPORTED;
    // an empty cache or table is nowhere
    if (!a->q || (a->pages && (!a->k_cache || !a->v_cache)) || (a->max_pages && !a->page_table) || !a->lengths || !a->out ||
        !a->workspace)
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
    // no row stands further than that from its sequence's first key, and the kernels may subtract it in 32 bits
    const int64_t reach = static_cast<int64_t>(a->max_pages) * a->page_size + kMaxRows;
    p.window = static_cast<int>(a->window < reach ? a->window : reach);
    p.cache_type = a->cache_type; p.scale = a->scale;
    if (sc) { p.slopes = sc->slopes; p.cap = sc->softcap; }
    const int rows_all = p.rows * p.group, es = p.cache_type == NVFP4_BF16 ? 2 : 1;
    TilePlan t;
    const bool tiles = host_variant() != 1 && p.group <= kMaxGroup && plan_tile(p.D, rows_all, &t);
    // units are counted in 31 bits: at least 16 keys each, one at least per sequence and column
    const int64_t most_units = (static_cast<int64_t>(a->max_pages) * a->page_size / 16 + 2) * a->seqs * a->kv_heads * t.chunks;
    // Whole 16-byte pieces of keys, and 16 keys of one page at a time; else a key per warp.
    if (tiles && most_units < (1ll << 31) && p.page % 16 == 0 && p.D * es % 16 == 0 &&
        aligned(p.cache[0], 16) && aligned(p.cache[1], 16) && p.page_stride[0] * es % 16 == 0 && p.page_stride[1] * es % 16 == 0 &&
        aligned(p.out, 8) && p.pages > 0 && p.page_stride[0] > 0 && p.page_stride[1] > 0 &&
        p.page_stride[0] * es < (1ll << 40) && p.page_stride[1] * es < (1ll << 40)) {
        const int grid = t.ctas_per_sm * sm_count();
        const Workspace w = workspace_of(t, sm_count(), p.D);
        p.chunks = t.chunks; p.chunk_rows = t.chunk_rows; p.columns = p.hk * t.chunks;
        char* base = static_cast<char*>(a->workspace);
        p.counters = reinterpret_cast<int*>(base);
        p.part_o = reinterpret_cast<float*>(base + w.part_o);
        p.part_ml = reinterpret_cast<float2*>(base + w.part_ml);
        p.row_blocks = t.row_blocks;
        p.wait_ns = host_wait_ns();
        p.group_inv = static_cast<uint32_t>(((1 << 24) + p.group - 1) / p.group);
        while ((4 << p.quad_log2) < p.D) ++p.quad_log2;
        p.page_tiles = p.page / 16;
        p.q_vec = aligned(p.q, 8) && p.q_ts % 4 == 0 && p.q_hs % 4 == 0;
        cudaStream_t st = static_cast<cudaStream_t>(stream);
        const bool scored = p.slopes || p.cap > 0.0f;
        if (p.cache_type == NVFP4_E2M1 || scored) {
            p.status = host_status_word();
            if (!p.status) return NVFP4_ERR_CUDA;
        }
        if (p.cache_type == NVFP4_E2M1) return scored ? launch_tiles_4bit_scored(t, p, grid, st) : launch_tiles_4bit(t, p, grid, st);
        if (scored) return launch_tiles_scored(t, p, grid, st);
        return p.cache_type == NVFP4_E4M3 ? dispatch_tile<NVFP4_E4M3, false>(t, p, grid, st)
                                          : dispatch_tile<NVFP4_BF16, false>(t, p, grid, st);
    }
    return launch(paged_attention_scalar_kernel, dim3(a->seqs * a->rows, a->q_heads), dim3(kScalarWarps * 32), 0,
                  static_cast<cudaStream_t>(stream), p);
}
