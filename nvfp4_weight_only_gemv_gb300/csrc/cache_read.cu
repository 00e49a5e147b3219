// Rows of a paged cache read back as bf16.
//
// For token t at position n = positions[t]: out[t, h] = bf16(code * block scale * scale[h]) (E2M1),
// bf16(code * scale[h]) (E4M3) or the value (bf16) of row n % page of page table[seq][n / page].
//
// Each value is moved once; the kernel is bound by that traffic for prompts, by latency for single tokens. (4 bits,
// 8192 tokens of 8 + 8 heads of 128 values: 12.2 us for 7.7 us of bytes, position, page and row being three trips one
// after the other; one token 2.4 us.)

#include "ops_common.cuh"

namespace nvfp4 {
namespace {

using namespace ops;

__device__ int g_read_status;

struct ReadParams {
    const void* cache[2];    // k, v
    const float* cache_scale[2];
    const int32_t* positions;
    const int32_t* seq_ids;  // NULL: token t belongs to sequence t / per_seq
    const int32_t* table;
    __nv_bfloat16* out[2];
    int64_t page_stride[2], table_stride;
    int64_t pieces;          // of all tokens' keys
    int T, hk, D, seqs, per_seq, pages, max_pages, page, cache_type;
    int head_pieces;         // of a head
};

// V neighbouring values of a row as they stand in the cache.
template <int V>
struct Piece {
    uint4 w[V == 16 ? 2 : 1];  // bf16: 32 bytes; E4M3: 16; E2M1: 8 of codes
    uint32_t block;            // E2M1: the scale's code
    __device__ __forceinline__ void load(const ReadParams& p, int which, int64_t page, int head, int slot, int d) {
        const char* const base = static_cast<const char*>(p.cache[which]);
        if (p.cache_type == NVFP4_E2M1) {
            const int64_t record = static_cast<int64_t>(head) * (p.page / kRecordKeys) + slot / kRecordKeys;
            const char* const rec = base + page * p.page_stride[which] + record * record_bytes(p.D);
            const int key = slot % kRecordKeys;
            const char* const codes = rec + key * (p.D / 2) + d / 2;
            if constexpr (V == 16) {
                const uint2 c = *reinterpret_cast<const uint2*>(codes);
                w[0].x = c.x; w[0].y = c.y;
            } else {
                w[0].x = static_cast<uint8_t>(*codes) >> 4 * (d & 1);
            }
            block = static_cast<uint8_t>(rec[8 * p.D + d / 16 * kRecordKeys + key]);
            return;
        }
        const int64_t at = page * p.page_stride[which] + (static_cast<int64_t>(head) * p.page + slot) * p.D + d;
        if (p.cache_type == NVFP4_E4M3) {
            if constexpr (V == 16) w[0] = *reinterpret_cast<const uint4*>(base + at);
            else w[0].x = static_cast<uint8_t>(base[at]);
        } else {
            if constexpr (V == 16) {
                w[0] = *reinterpret_cast<const uint4*>(base + 2 * at);
                w[1] = *reinterpret_cast<const uint4*>(base + 2 * at + 16);
            } else {
                w[0].x = *reinterpret_cast<const uint16_t*>(base + 2 * at);
            }
        }
    }
    __device__ __forceinline__ void store(const ReadParams& p, float scale, __nv_bfloat16* out) const {
        if (p.cache_type == NVFP4_BF16) {  // as it stands
            if constexpr (V == 16) {
                *reinterpret_cast<uint4*>(out) = w[0];
                *reinterpret_cast<uint4*>(out + 8) = w[1];
            } else {
                *reinterpret_cast<uint16_t*>(out) = static_cast<uint16_t>(w[0].x);
            }
            return;
        }
        const uint32_t words[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
        const float b = p.cache_type == NVFP4_E2M1 ? e4m3_value(block) : 1.0f;
        uint32_t halves[V == 16 ? 8 : 1];
        if constexpr (V == 16) {
            if (p.cache_type == NVFP4_E2M1) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint32_t h4[4];
                    e2m1x8_f16x2(words[i], h4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) halves[4 * i + e] = h4[e];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) halves[i] = e4m3x2_f16x2(words[i / 2] >> 16 * (i & 1));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&halves[4 * i + e]));
                    y[e] = pack_bf16(f.x * b * scale, f.y * b * scale);
                }
                *reinterpret_cast<uint4*>(out + 8 * i) = make_uint4(y[0], y[1], y[2], y[3]);
            }
        } else {
            uint32_t h4[4];
            e2m1x8_f16x2(words[0], h4);
            const uint32_t code = p.cache_type == NVFP4_E2M1 ? h4[0] : e4m3x2_f16x2(words[0]);
            *out = __float2bfloat16_rn(__half2float(__ushort_as_half(static_cast<unsigned short>(code & 0xffffu))) * b * scale);
        }
    }
};

// One thread takes V neighbouring values of a key and the same of its value: 16 where rows are whole blocks on their
// boundaries, else one.
template <int V>
__global__ void __launch_bounds__(128) cache_read_kernel(const __grid_constant__ ReadParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (at >= p.pieces) return;
    const int per_token = p.hk * p.head_pieces;
    const int t = p.pieces <= INT32_MAX ? static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(per_token)) : static_cast<int>(at / per_token);
    const int i = static_cast<int>(at - static_cast<int64_t>(t) * per_token), h = i / p.head_pieces, d = (i - h * p.head_pieces) * V;
    const int n = p.positions[t];
    int64_t page = -1;
    if (n >= 0) {
        const int seq = p.seq_ids ? p.seq_ids[t] : t / p.per_seq, pi = n / p.page;
        if (seq >= 0 && seq < p.seqs && pi < p.max_pages) page = p.table[seq * p.table_stride + pi];
        if (page < 0 || page >= p.pages) {
            page = -1;
            atomicOr(&g_read_status, NVFP4_DEV_BAD_PAGE);
        }
    }
    const int64_t to = (static_cast<int64_t>(t) * p.hk + h) * p.D + d;
    if (page < 0) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __nv_bfloat16* const out = p.out[which] + to;
            if constexpr (V == 16) reinterpret_cast<uint4*>(out)[0] = reinterpret_cast<uint4*>(out)[1] = make_uint4(0, 0, 0, 0);
            else *out = __float2bfloat16_rn(0.0f);
        }
        return;
    }
    Piece<V> piece[2];
    float scale[2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        piece[which].load(p, which, page, h, n % p.page, d);
        scale[which] = p.cache_scale[which] ? p.cache_scale[which][h] : 1.0f;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) piece[which].store(p, scale[which], p.out[which] + to);
}

cudaError_t read_status(int* bits) {
    const int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, g_read_status, sizeof(int));
    return e != cudaSuccess || *bits == 0 ? e : cudaMemcpyToSymbol(g_read_status, &zero, sizeof(int));
}
const bool g_registered = register_status(read_status);

}  // namespace
}  // namespace nvfp4

extern "C" nvfp4_status nvfp4_cache_read(const nvfp4_cache_read_args* a, void* stream) {
    using namespace nvfp4;
    using namespace nvfp4::ops;
    if (!a) return NVFP4_ERR_NULL;
    if (a->tokens < 0 || a->kv_heads < 0 || a->head_dim < 0 || a->seqs < 0 || a->pages < 0 || a->max_pages < 0 || a->page_size < 1)
        return NVFP4_ERR_SHAPE;
    if ((a->cache_type != NVFP4_BF16 && a->cache_type != NVFP4_E4M3 && a->cache_type != NVFP4_E2M1) ||
        (a->cache_type == NVFP4_BF16 && (a->k_scale || a->v_scale)))
        return NVFP4_ERR_DTYPE;
    if (a->cache_type == NVFP4_E2M1 && (a->head_dim % 16 || a->page_size % kRecordKeys)) return NVFP4_ERR_SHAPE;
    if (a->tokens == 0 || a->kv_heads == 0 || a->head_dim == 0) return NVFP4_OK;
    if (a->head_dim > 1024 || a->kv_heads > 32767 || static_cast<int64_t>(a->max_pages) * a->page_size > (1 << 24))
        return NVFP4_ERR_UNSUPPORTED;
    // an empty cache or table is nowhere
    if (!a->positions || !a->k_out || !a->v_out || (a->pages && (!a->k_cache || !a->v_cache)) || (a->max_pages && !a->page_table))
        return NVFP4_ERR_NULL;
    if (a->seqs == 0 || (!a->seq_ids && a->tokens % a->seqs)) return NVFP4_ERR_SHAPE;
    ReadParams p{};
    p.cache[0] = a->k_cache; p.cache[1] = a->v_cache;
    p.cache_scale[0] = a->k_scale; p.cache_scale[1] = a->v_scale;
    p.positions = a->positions; p.seq_ids = a->seq_ids; p.table = a->page_table;
    p.out[0] = static_cast<__nv_bfloat16*>(a->k_out); p.out[1] = static_cast<__nv_bfloat16*>(a->v_out);
    p.page_stride[0] = a->k_page_stride; p.page_stride[1] = a->v_page_stride; p.table_stride = a->table_stride;
    p.T = a->tokens; p.hk = a->kv_heads; p.D = a->head_dim; p.seqs = a->seqs;
    p.per_seq = (a->tokens + a->seqs - 1) / a->seqs;
    p.pages = a->pages; p.max_pages = a->max_pages; p.page = a->page_size; p.cache_type = a->cache_type;
    // 16 values a thread: pieces of 8 (E2M1) or 16 bytes on their boundaries
    const int piece = p.cache_type == NVFP4_E2M1 ? 8 : 16, elements = p.cache_type == NVFP4_BF16 ? 8 : piece;
    bool wide = host_variant() != 1 && p.D % 16 == 0;
    for (int i = 0; i < 2; ++i)
        wide = wide && aligned(p.cache[i], piece) && p.page_stride[i] % elements == 0 && aligned(p.out[i], 16);
    p.head_pieces = wide ? p.D / 16 : p.D;
    p.pieces = static_cast<int64_t>(p.T) * p.hk * p.head_pieces;
    const int64_t ctas = (p.pieces + 127) / 128;
    if (ctas > INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(ctas));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return wide ? launch(cache_read_kernel<16>, grid, dim3(128), 0, st, p) : launch(cache_read_kernel<1>, grid, dim3(128), 0, st, p);
}
