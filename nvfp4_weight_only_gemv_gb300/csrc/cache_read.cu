// Rows of a paged cache read back as bf16.
//
// For token t at position n = positions[t]: out[t, h] = bf16(code * block scale * scale[h]) (E2M1),
// bf16(code * scale[h]) (E4M3) or the value (bf16) of row n % page of page table[seq][n / page]; code * block scale is exact,
// its product with a head's scale fp32's.
//
// Each value is moved once; the kernel is bound by that traffic for prompts, by latency for single tokens. (8192 tokens of
// 8 + 8 heads of 128 values, back to back in a graph: 9.6 us in 4 bits for 6.3 us of bytes, E4M3 10.2 for 7.4, bf16 12.6 for
// 9.9, position, page and row being three trips one after the other; one token 2.0 us of any.)

#include "ops_common.cuh"

namespace nvfp4 {
namespace {

using namespace ops;

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
    int* status;             // see host_status_word
    int head_pieces;         // of a head
    int sectors;             // the outputs begin on 32-byte boundaries
};

// 32 bytes, a whole sector at once where they lie on its boundary: in two halves a warp's stores touch every sector twice.
__device__ __forceinline__ void store32(__nv_bfloat16* out, bool sector, uint4 a, uint4 b) {
    if (sector) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     ::"l"(out), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
    } else {
        reinterpret_cast<uint4*>(out)[0] = a;
        reinterpret_cast<uint4*>(out)[1] = b;
    }
}

// Sixteen neighbouring values of a row as they stand in a cache of type C, or one in any.
template <int C>
struct Piece {
    uint4 w[C == NVFP4_BF16 ? 2 : 1];  // bf16: 32 bytes; E4M3: 16; E2M1: 8 of codes
    uint32_t block;                    // E2M1: the scale's code
    __device__ __forceinline__ void load(const ReadParams& p, int which, int64_t page, int head, int slot, int d) {
        const char* const base = static_cast<const char*>(p.cache[which]) + page * p.page_stride[which] * (C == NVFP4_BF16 ? 2 : 1);
        if constexpr (C == NVFP4_E2M1) {
            const int key = slot % kRecordKeys;
            const char* const rec = base + (static_cast<int64_t>(head) * (p.page / kRecordKeys) + slot / kRecordKeys) * record_bytes(p.D);
            const uint2 c = *reinterpret_cast<const uint2*>(rec + key * (p.D / 2) + d / 2);
            w[0].x = c.x; w[0].y = c.y;
            block = static_cast<uint8_t>(rec[8 * p.D + d + key]);
        } else {
            const char* const at = base + ((static_cast<int64_t>(head) * p.page + slot) * p.D + d) * (C == NVFP4_BF16 ? 2 : 1);
            w[0] = *reinterpret_cast<const uint4*>(at);
            if constexpr (C == NVFP4_BF16) w[1] = *reinterpret_cast<const uint4*>(at + 16);
        }
    }
    __device__ __forceinline__ void store(float scale, __nv_bfloat16* out, bool sector) const {
        if constexpr (C == NVFP4_BF16) {  // as it stands
            store32(out, sector, w[0], w[1]);
        } else {
            uint4 out2[2];
            const uint32_t words[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
            const float b = C == NVFP4_E2M1 ? e4m3_value(block) : 1.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t halves[4], y[4];
                if constexpr (C == NVFP4_E2M1) {
                    e2m1x8_f16x2(words[i], halves);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) halves[e] = e4m3x2_f16x2(words[2 * i + e / 2] >> 16 * (e & 1));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&halves[e]));
                    y[e] = pack_bf16(f.x * b * scale, f.y * b * scale);
                }
                out2[i] = make_uint4(y[0], y[1], y[2], y[3]);
            }
            store32(out, sector, out2[0], out2[1]);
        }
    }
};

// The page of token t's row and its slot there; -1 for padding, and (with a status bit) where there is no such place.
__device__ __forceinline__ int64_t page_of(const ReadParams& p, int t, int& slot) {
    const int n = p.positions[t];
    if (n < 0) return -1;
    const int seq = p.seq_ids ? p.seq_ids[t] : t / p.per_seq, pi = n / p.page;
    slot = n - pi * p.page;
    if (seq >= 0 && seq < p.seqs && pi < p.max_pages) {
        const int page = p.table[seq * p.table_stride + pi];
        if (page >= 0 && page < p.pages) return page;
    }
    atomicOr(p.status, NVFP4_DEV_BAD_PAGE);
    return -1;
}

// One value a thread: any head size and alignment.
__global__ void __launch_bounds__(128) cache_read_scalar_kernel(const __grid_constant__ ReadParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (at >= 2 * p.pieces) return;
    const int which = at >= p.pieces;
    const int64_t to = at - which * p.pieces;
    const int per_token = p.hk * p.D, t = static_cast<int>(to / per_token), i = static_cast<int>(to - static_cast<int64_t>(t) * per_token);
    const int h = i / p.D, d = i - h * p.D;
    int slot = 0;
    const int64_t page = page_of(p, t, slot);
    __nv_bfloat16* const out = p.out[which] + to;
    if (page < 0) {
        *out = __float2bfloat16_rn(0.0f);
        return;
    }
    const float scale = p.cache_scale[which] ? p.cache_scale[which][h] : 1.0f;
    if (p.cache_type == NVFP4_E2M1) {
        const int64_t record = static_cast<int64_t>(h) * (p.page / kRecordKeys) + slot / kRecordKeys;
        const uint8_t* const rec = static_cast<const uint8_t*>(p.cache[which]) + page * p.page_stride[which] + record * record_bytes(p.D);
        const int key = slot % kRecordKeys;
        uint32_t h2[4];
        e2m1x8_f16x2(rec[key * (p.D / 2) + d / 2], h2);
        const float v = __half2float(__ushort_as_half(static_cast<unsigned short>(d & 1 ? h2[0] >> 16 : h2[0] & 0xffffu)));
        *out = __float2bfloat16_rn(v * e4m3_value(rec[8 * p.D + d / 16 * kRecordKeys + key]) * scale);
        return;
    }
    const int64_t from = page * p.page_stride[which] + (static_cast<int64_t>(h) * p.page + slot) * p.D + d;
    if (p.cache_type == NVFP4_E4M3) *out = __float2bfloat16_rn(e4m3_value(static_cast<const uint8_t*>(p.cache[which])[from]) * scale);
    else *out = static_cast<const __nv_bfloat16*>(p.cache[which])[from];
}

// One thread takes 16 neighbouring values of a key and the same of its value. (4 bits, 8192 tokens of 8 + 8 heads of
// 128 values, us by single launches: 10.0; with stores of 16 bytes 12.2; two or four such pairs a thread 12.3 and 13.5, 8 values 14.2.)
template <int C>
__global__ void __launch_bounds__(128) cache_read_kernel(const __grid_constant__ ReadParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x;
    if (at >= p.pieces) return;
    const int per_token = p.hk * p.head_pieces;
    const int t = at >> 32 ? static_cast<int>(at / per_token) : static_cast<int>(static_cast<uint32_t>(at) / static_cast<uint32_t>(per_token));
    const int i = static_cast<int>(at - static_cast<int64_t>(t) * per_token), h = i / p.head_pieces, d = (i - h * p.head_pieces) * 16;
    int slot = 0;
    const int64_t page = page_of(p, t, slot);
    __nv_bfloat16* const out[2] = {p.out[0] + at * 16, p.out[1] + at * 16};  // pieces lie as the output does
    if (page < 0) {
        for (int which = 0; which < 2; ++which) store32(out[which], p.sectors, make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0));
        return;
    }
    Piece<C> piece[2];
    float scale[2];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        piece[which].load(p, which, page, h, slot, d);
        scale[which] = p.cache_scale[which] ? p.cache_scale[which][h] : 1.0f;
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) piece[which].store(scale[which], out[which], p.sectors);
}

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
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int64_t ctas = ((wide ? 1 : 2) * p.pieces + 127) / 128;
    if (ctas > INT32_MAX) return NVFP4_ERR_UNSUPPORTED;
    p.status = host_status_word();
    if (!p.status) return NVFP4_ERR_CUDA;
    p.sectors = aligned(p.out[0], 32) && aligned(p.out[1], 32);
    const auto kernel = !wide ? cache_read_scalar_kernel : p.cache_type == NVFP4_E2M1 ? cache_read_kernel<NVFP4_E2M1>
                      : p.cache_type == NVFP4_E4M3 ? cache_read_kernel<NVFP4_E4M3> : cache_read_kernel<NVFP4_BF16>;
    return launch(kernel, dim3(static_cast<unsigned>(ctas)), dim3(128), 0, st, p);
}
