// Rotary positions of q and k, and the append of k and v to a paged cache.
//
// For token t at position n = positions[t], per head of q and k (v is only appended):
//   u      = x / sqrt(mean(x^2) + eps) * w            (per-head norm; left out without weights)
//   y[a_i] = u[a_i] c_i - u[b_i] s_i,  y[b_i] = u[b_i] c_i + u[a_i] s_i,   i < half
//   c_i, s_i = mscale * cos, sin(n * inv_freq[i])
//   (a_i, b_i) = (i, i + half) or, interleaved, (2i, 2i + 1); the head's other values pass through
// q goes to q_out in bf16, k and v to row n % page of page table[seq][n / page] of the cache
// [pages, kv heads, page, D], in bf16, as E4M3(value / scale[kv head]), or in 4 bits: of 16 neighbours
// t = value / scale[kv head] a block scale b = E4M3(max|t| / 6) and the codes E2M1(t / b).
//
// The kernel moves each value once and is bound by that traffic for prompts, by latency for
// single tokens.

#include "ops_common.cuh"

namespace nvfp4 {
namespace {

using namespace ops;

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
    int norm_type, interleaved, cache_type;
    float mscale, eps, one_over_d;
    int* status;             // see host_status_word
    int shares, lanes_log2;  // vector kernel: warps per token, lanes per head
};

// cos and sin of n * f for a whole n below 2^24. f / pi is taken as a sum of two floats (1 / pi as
// 0x1.45f306p-2 + 0x1.b9391p-27), n times its first part exactly as another such sum, and whole turns
// leave that without an error, so the angle is as exact at position 10^7 as at 10: about 2^-23 off. The
// product alone, rounded to fp32, would be off by half a unit in its last place, 0.03 at n f = 10^6.
__device__ __forceinline__ float2 cos_sin(int n, float f) {
    const float c1 = 0x1.45f306p-2f, c2 = 0x1.b9391p-27f;
    const float hi = f * c1, lo = fmaf(f, c2, fmaf(f, c1, -hi));
    const float nf = static_cast<float>(n);
    const float p = nf * hi, e = fmaf(nf, lo, fmaf(nf, hi, -p));
    const float r = (p - 2.0f * rintf(0.5f * p)) + e;  // half turns, within one of zero
    float s, c;
    sincospif(r, &s, &c);
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
    atomicOr(p.status, NVFP4_DEV_BAD_PAGE);
    return false;
}

// The E4M3 code of a block's scale from the bits of its largest magnitude `top`: the fp32 quotient by 6, rounded to
// nearest, at most 448; NaN where top is one.
__device__ __forceinline__ uint32_t block_scale(uint32_t top) {
    if (top > 0x7f800000u) return 0x7fu;
    const float t = fminf(__uint_as_float(top), 8192.0f), inv = 1.0f / 6.0f;  // 8192 / 6 is far beyond 448
    return pack_e4m3(put_right(t * inv, t, 6.0f, inv), 0.0f) & 0xffu;
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
    auto turned = [&](int d) {
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
        return y;
    };
    if (part > 0 && p.cache_type == NVFP4_E2M1) {
        // 16 lanes hold a block: its largest magnitude (a NaN's is the largest of all), its scale, its codes
        const float* const sc = p.cache_scale[part - 1];
        const int64_t record = static_cast<int64_t>(h) * (p.page / kRecordKeys) + at.slot / kRecordKeys;
        uint8_t* const rec = static_cast<uint8_t*>(p.cache[part - 1]) + at.page * p.page_stride[part - 1] + record * record_bytes(p.D);
        const int key = at.slot % kRecordKeys;
        for (int first = 0; first < p.D; first += 128) {  // every lane goes through the shuffles
            const int d = first + tid;
            const float v = d < p.D ? turned(d) / (sc ? sc[h] : 1.0f) : 0.0f;
            uint32_t top = __float_as_uint(v) & 0x7fffffffu;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t b = block_scale(top);
            const float bs = e4m3_value(b), mine = bs == 0.0f ? 0.0f : v / bs;
            const float pair[8] = {mine, __shfl_xor_sync(0xffffffffu, mine, 1), 0, 0, 0, 0, 0, 0};
            if (d >= p.D) continue;
            if ((d & 1) == 0) rec[key * (p.D / 2) + d / 2] = static_cast<uint8_t>(pack_e2m1x8(pair));
            if (d % 16 == 0) rec[8 * p.D + d + key] = static_cast<uint8_t>(b);
        }
        return;
    }
    for (int d = tid; d < p.D; d += 128) {
        const float y = turned(d);
        if (part == 0) {
            p.q_out[(static_cast<int64_t>(t) * p.hq + h) * p.D + d] = __float2bfloat16_rn(ok ? y : 0.0f);
        } else {
            const int64_t to = at.page * p.page_stride[part - 1] + (static_cast<int64_t>(h) * p.page + at.slot) * p.D + d;
            if (p.cache_type == NVFP4_E4M3) {
                const float* sc = p.cache_scale[part - 1];
                static_cast<uint8_t*>(p.cache[part - 1])[to] = static_cast<uint8_t>(pack_e4m3(y / (sc ? sc[h] : 1.0f), 0.0f));
            } else {
                static_cast<__nv_bfloat16*>(p.cache[part - 1])[to] = __float2bfloat16_rn(y);
            }
        }
    }
}

// Vector kernel: a lane holds 2 V values of a head as two vectors, chosen so that both members of each
// rotated pair are its own: in halves, values V i.. and half + V i..; interleaved, or beyond the
// rotary part, 2 V neighbours. D / (2 V) lanes make a head (V = 8: 16-byte pieces of bf16). A warp
// takes a token, or a share of its heads where tokens are few, on its own: it forms the token's
// cosines and sines once, keeps those of its pairs in registers, and walks through the heads of q, k
// and v by constant steps with the next vectors on their way. (One pair after the other, the places
// found per head, and cosines shared by a CTA behind a barrier: 8192 tokens of 32 + 8 + 8 heads took
// 64 us; this way 39.5, 5.1 TB/s. Bound by latency: five CTAs an SM hold 40 KB of vectors in flight.)
constexpr int kThreads = 128;

template <typename XT, int V>
struct Piece;  // V consecutive values as loaded
template <int V>
struct Piece<float, V> {
    float4 w[V / 4];
    __device__ __forceinline__ void load(const float* p) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + 4 * i);
    }
    __device__ __forceinline__ void widen(float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) { v[4 * i] = w[i].x; v[4 * i + 1] = w[i].y; v[4 * i + 2] = w[i].z; v[4 * i + 3] = w[i].w; }
    }
};
template <int V>
struct Piece<__nv_bfloat16, V> {
    uint32_t w[V / 2];
    __device__ __forceinline__ void load(const __nv_bfloat16* p) {
        if constexpr (V == 8) {
            const uint4 q = *reinterpret_cast<const uint4*>(p);
            w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
        } else {
            const uint2 q = *reinterpret_cast<const uint2*>(p);
            w[0] = q.x; w[1] = q.y;
        }
    }
    __device__ __forceinline__ void widen(float (&v)[V]) const {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) unpack_bf16(w[i], v[2 * i], v[2 * i + 1]);
    }
};

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float (&v)[V]) {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) w[i] = pack_e4m3(v[4 * i], v[4 * i + 1]) | pack_e4m3(v[4 * i + 2], v[4 * i + 3]) << 16;
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// x / s for E4M3 from inv = 1 / s. A quotient of 512 and more only has to stay beyond 448, infinities with it. (A
// division per value took 8192 tokens of 32 + 8 + 8 heads from 45.7 to 49.8 us, this does not.)
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    return put_right(fminf(fmaxf(x * inv, -512.0f), 512.0f), x, s, inv);
}

// Scales of which 1 / scale might not be normal are taken times a power of two, with the values; by an infinite one what is
// finite becomes zero.
template <int V>
__device__ __forceinline__ void lift_scale(float& scale, float (&a)[V], float (&b)[V]) {
    if (fabsf(scale) >= 0x1p-100f && fabsf(scale) <= 0x1p100f) return;
    const bool infinite = fabsf(scale) == INFINITY;
    const float lift = fabsf(scale) < 1.0f ? 0x1p64f : infinite ? 0.0f : 0x1p-64f;
    scale = infinite ? copysignf(1.0f, scale) : scale * lift;
#pragma unroll
    for (int e = 0; e < V; ++e) { a[e] *= lift; b[e] *= lift; }
}

// Beyond any block's largest value that a scale can still express.
constexpr float kFar = 8192.0f;

// x / s for |x / s| up to `most` and something beyond for what lies beyond; as put_right, and a zero keeps its sign.
__device__ __forceinline__ float quotient_to(float most, float x, float s, float inv) {
    const float q = fminf(fmaxf(x * inv, -most), most);
    return fmaf(fmaf(q, s, -x), -inv, q);
}

// The E2M1 codes of eight (or, in the low half, four) values of a block whose scale stands for b.
template <int V>
__device__ __forceinline__ uint32_t block_codes(const float (&x)[V], float b) {
    if (b == 0.0f) return 0u;
    // b has 4 bits, so a quotient lies 2^-28 of itself and more from the middle of two floats, and what the correction
    // leaves of a reciprocal that is a unit off, 2^-46, does not reach it
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(b));
    float v[8] = {};
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = quotient_to(8.0f, x[e], b, inv);
    return pack_e2m1x8(v);
}

// F4: a cache of 4 bits. With V = 8 a lane's vectors are halves of two blocks, whose other halves its neighbours have, or, where
// pairs are neighbours or do not turn, one block; with V = 4, quarters of any, whose largest values meet in shared memory. (8192 tokens of 32 + 8 + 8 heads: 46.3 us, 3.8 TB/s, where bf16
// takes 39.1 for more bytes: the codes' arithmetic is 2 to 3 us of that, the rest latency at the same 27 % of the warps, with more
// state: 28 bytes of spills at 96 registers. A block's scale stored or not and quotients without clamps made no difference; 128 registers,
// 80, cosines read from shared memory each time, rows prefetched into L2 took 52, 58, 53, 51.)
template <typename XT, int V, bool F4>
__global__ void __launch_bounds__(kThreads, 5) rope_append_kernel(const __grid_constant__ AppendParams p) {
    constexpr int kDepth = sizeof(XT) == 2 ? 2 : 1;   // heads requested ahead
    extern __shared__ __align__(16) float2 cs_all[];  // [warps][half]
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int unit = blockIdx.x * (kThreads / 32) + warp;
    const int tok = unit / p.shares, share = unit - tok * p.shares;
    const int lanes = 1 << p.lanes_log2, hpi = 32 >> p.lanes_log2;  // heads at a time
    const int i = lane & (lanes - 1), sub = lane >> p.lanes_log2;
    // offsets of the lane's two vectors
    const bool turns = V * i < p.half, halves = turns && !p.interleaved, live = 2 * V * i < p.D;
    const int oa = halves ? V * i : 2 * V * i, ob = halves ? p.half + V * i : 2 * V * i + V;
    // this share's steps out of the token's: those of q, then of k, then of v
    const int sq = (p.hq + hpi - 1) >> (5 - p.lanes_log2), sk = (p.hk + hpi - 1) >> (5 - p.lanes_log2), all = sq + 2 * sk;
    const int begin = all * share / p.shares, end = all * (share + 1) / p.shares;
    pdl_wait();
    if (tok >= p.T) return;
    const int n = p.positions[tok];
    float2* const cs = cs_all + warp * p.half;
    Place at{0, 0};
    const bool placed = end > sq && place_of(p, tok, n, at);
    float c[V], s[V];
    if (begin < sq + sk && p.half > 0) {
        for (int j = lane; j < p.half; j += 32) {
            const float2 v = cos_sin(n < 0 ? 0 : n, p.inv_freq[j]);
            cs[j] = make_float2(v.x * p.mscale, v.y * p.mscale);
        }
        __syncwarp();
        if (turns) {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float4 v = *reinterpret_cast<const float4*>(cs + V * i + e);
                c[e] = v.x; s[e] = v.y; c[e + 1] = v.z; s[e + 1] = v.w;
            }
        }
    }
#pragma unroll
    for (int part = 0; part < 3; ++part) {
        const int first = part == 0 ? 0 : part == 1 ? sq : sq + sk, heads = part == 0 ? p.hq : p.hk;
        const int from = max(begin, first), to = min(end, first + (part == 0 ? sq : sk));
        if (from >= to || (part > 0 && !placed)) continue;
        int h = (from - first) * hpi + sub;
        const XT* x = static_cast<const XT*>(p.x[part]) + tok * p.ts[part] + h * p.hs[part];
        const int64_t x_step = hpi * p.hs[part];
        const void* const w = part == 0 ? p.q_norm : part == 1 ? p.k_norm : nullptr;
        // lanes beyond the head hold zeros throughout: the norm's sum counts on it
        Piece<XT, V> na[kDepth], nb[kDepth];
        int ahead = h;
#pragma unroll
        for (int d = 0; d < kDepth; ++d, ahead += hpi, x += x_step) {
            na[d] = nb[d] = Piece<XT, V>{};
            if (live && ahead < heads) { na[d].load(x + oa); nb[d].load(x + ob); }
        }
        float wa[V], wb[V];
        if (part < 2 && w && live) {
            if (p.norm_type == NVFP4_F32) {
                Piece<float, V> q;
                q.load(static_cast<const float*>(w) + oa); q.widen(wa);
                q.load(static_cast<const float*>(w) + ob); q.widen(wb);
            } else {
                Piece<__nv_bfloat16, V> q;
                q.load(static_cast<const __nv_bfloat16*>(w) + oa); q.widen(wa);
                q.load(static_cast<const __nv_bfloat16*>(w) + ob); q.widen(wb);
            }
        }
        // the head's row in the output or the cache, bytes
        const bool records = F4 && part > 0;
        const int64_t between = part == 0 ? p.D : records ? p.page / kRecordKeys * record_bytes(p.D) : static_cast<int64_t>(p.page) * p.D;
        const int64_t row = (part == 0 ? static_cast<int64_t>(tok) * p.hq * p.D
                                       : at.page * p.page_stride[part - 1] + (records ? at.slot / kRecordKeys * record_bytes(p.D)
                                                                                      : static_cast<int64_t>(at.slot) * p.D)) + h * between;
        const int y_size = part > 0 && p.cache_type != NVFP4_BF16 ? 1 : 2;
        char* y = (part == 0 ? reinterpret_cast<char*>(p.q_out) : static_cast<char*>(p.cache[part - 1])) + row * y_size;
        const int64_t y_step = hpi * between * y_size;
        auto head = [&](Piece<XT, V>& ra, Piece<XT, V>& rb) {
            // requested, and inverted, ahead of the values' arithmetic
            const float* const by = F4 && part > 0 ? p.cache_scale[part - 1] : nullptr;
            float scale4 = by && h < heads ? by[h] : 1.0f;
            float a[V], b[V];
            ra.widen(a);
            rb.widen(b);
            if (live && ahead < heads) { ra.load(x + oa); rb.load(x + ob); }
            ahead += hpi;
            x += x_step;
            if (part < 2 && w) {
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) sum = fmaf(a[e], a[e], fmaf(b[e], b[e], sum));
                for (int o = 1; o < lanes; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float rstd = rsqrtf(fmaf(sum, p.one_over_d, p.eps));
#pragma unroll
                for (int e = 0; e < V; ++e) { a[e] *= rstd * wa[e]; b[e] *= rstd * wb[e]; }
            }
            if (part < 2 && turns) {
                if (halves) {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float u = a[e] * c[e] - b[e] * s[e];
                        b[e] = b[e] * c[e] + a[e] * s[e];
                        a[e] = u;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float* const u = 2 * e < V ? a + 2 * e : b + 2 * e - V;
                        const float v = u[0] * c[e] - u[1] * s[e];
                        u[1] = u[1] * c[e] + u[0] * s[e];
                        u[0] = v;
                    }
                }
            }
            if (part == 0 && n < 0) {
#pragma unroll
                for (int e = 0; e < V; ++e) a[e] = b[e] = 0.0f;
            }
            if constexpr (F4) {
                if (part > 0) {
                    if (by) {
                        lift_scale(scale4, a, b);
                        const float inv = 1.0f / scale4;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            a[e] = quotient_to(kFar, a[e], scale4, inv);
                            b[e] = quotient_to(kFar, b[e], scale4, inv);
                        }
                    }
                    uint32_t ta = 0, tb = 0;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        ta = max(ta, __float_as_uint(a[e]) & 0x7fffffffu);
                        tb = max(tb, __float_as_uint(b[e]) & 0x7fffffffu);
                    }
                    if constexpr (V == 4) {
                        // the head's vectors in order: this lane's are the va-th and the vb-th
                        const int va = oa / V, vb = ob / V, row0 = sub * 2 * lanes;
                        uint32_t* const tops = reinterpret_cast<uint32_t*>(cs_all + kThreads / 32 * p.half) + warp * 64;
                        if (live) { tops[row0 + va] = ta; tops[row0 + vb] = tb; }
                        __syncwarp();
                        if (live && h < heads) {
                            auto top_of = [&](int vec) {
                                const uint4 t4 = *reinterpret_cast<const uint4*>(tops + row0 + (vec & ~3));
                                return max(max(t4.x, t4.y), max(t4.z, t4.w));
                            };
                            const uint32_t ba = block_scale(top_of(va)), bb = block_scale(top_of(vb));
                            const int key = at.slot % kRecordKeys;
                            uint8_t* const rec = reinterpret_cast<uint8_t*>(y);
                            uint8_t* const codes = rec + key * (p.D >> 1);
                            *reinterpret_cast<uint16_t*>(codes + (oa >> 1)) = static_cast<uint16_t>(block_codes(a, e4m3_value(ba)));
                            *reinterpret_cast<uint16_t*>(codes + (ob >> 1)) = static_cast<uint16_t>(block_codes(b, e4m3_value(bb)));
                            if (va % 4 == 0) rec[8 * p.D + oa + key] = static_cast<uint8_t>(ba);
                            if (vb % 4 == 0) rec[8 * p.D + ob + key] = static_cast<uint8_t>(bb);
                        }
                        __syncwarp();
                        h += hpi;
                        y += y_step;
                        return;
                    }
                    uint32_t na = __shfl_xor_sync(0xffffffffu, ta, 1), nb = __shfl_xor_sync(0xffffffffu, tb, 1);
                    if (p.half & 8) {  // where the halves meet, a block has the last lane's first and the first lane's second vector
                        const uint32_t first = __shfl_sync(0xffffffffu, tb, lane - i), last = __shfl_sync(0xffffffffu, ta, lane - i + (p.half >> 3) - 1);
                        const uint32_t mid = __shfl_sync(0xffffffffu, tb, i == 0 ? lane : i & 1 ? lane + 1 : lane - 1);
                        if (i == (p.half >> 3) - 1) na = first;
                        nb = i == 0 ? last : mid;
                    }
                    const uint32_t ba = block_scale(max(ta, halves ? na : tb)), bb = halves ? block_scale(max(tb, nb)) : ba;
                    if (live && h < heads) {
                        const int key = at.slot % kRecordKeys;
                        uint8_t* const rec = reinterpret_cast<uint8_t*>(y);
                        uint8_t* const codes = rec + key * (p.D >> 1);
                        *reinterpret_cast<uint32_t*>(codes + (oa >> 1)) = block_codes(a, e4m3_value(ba));
                        *reinterpret_cast<uint32_t*>(codes + (ob >> 1)) = block_codes(b, e4m3_value(bb));
                        // one lane stores a block's scale: of two neighbours the first that of a, the second that of b
                        const bool second = halves && (i & 1);
                        rec[8 * p.D + ((second ? ob : oa) & ~15) + key] = static_cast<uint8_t>(second ? bb : ba);
                    }
                    h += hpi;
                    y += y_step;
                    return;
                }
            }
            if (live && h < heads) {
                if (part > 0 && p.cache_type == NVFP4_E4M3) {
                    const float* const sc = p.cache_scale[part - 1];
                    if (sc) {
                        float scale = sc[h];
                        lift_scale(scale, a, b);
                        const float inv = 1.0f / scale;
#pragma unroll
                        for (int e = 0; e < V; ++e) { a[e] = quotient(a[e], scale, inv); b[e] = quotient(b[e], scale, inv); }
                    }
                    store_codes(reinterpret_cast<uint8_t*>(y) + oa, a);
                    store_codes(reinterpret_cast<uint8_t*>(y) + ob, b);
                } else {
                    store_vec(reinterpret_cast<__nv_bfloat16*>(y) + oa, a);
                    store_vec(reinterpret_cast<__nv_bfloat16*>(y) + ob, b);
                }
            }
            h += hpi;
            y += y_step;
        };
        for (int k = from; k < to; k += kDepth) {
            head(na[0], nb[0]);
            if constexpr (kDepth > 1) {
                if (k + 1 < to) head(na[1], nb[1]);
            }
        }
    }
}

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
    if ((a->x_type != NVFP4_F32 && a->x_type != NVFP4_BF16) || (a->cache_type != NVFP4_BF16 && a->cache_type != NVFP4_E4M3 && a->cache_type != NVFP4_E2M1) ||
        (a->cache_type == NVFP4_BF16 && (a->k_scale || a->v_scale)) ||
        ((a->q_norm || a->k_norm) && a->norm_type != NVFP4_F32 && a->norm_type != NVFP4_BF16))
        return NVFP4_ERR_DTYPE;
    if (a->cache_type == NVFP4_E2M1 && (a->head_dim % 16 || a->page_size % kRecordKeys)) return NVFP4_ERR_SHAPE;
    if (a->tokens == 0 || a->head_dim == 0 || hq + a->kv_heads == 0) return NVFP4_OK;
    if (a->head_dim > 1024 || static_cast<int64_t>(hq) + 2 * static_cast<int64_t>(a->kv_heads) > 65535 ||
        static_cast<int64_t>(a->max_pages) * a->page_size > (1 << 24))
        return NVFP4_ERR_UNSUPPORTED;
    if (!a->positions || (a->rotary_half && !a->inv_freq) || (hq && !a->q_out) ||
        (a->kv_heads && (!a->k || !a->v || (a->pages && (!a->k_cache || !a->v_cache)) || (a->max_pages && !a->page_table))))
        return NVFP4_ERR_NULL;  // (an empty cache or table is nowhere)
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
    p.norm_type = a->norm_type; p.interleaved = a->interleaved; p.cache_type = a->cache_type;
    p.mscale = a->mscale; p.eps = a->eps;
    p.status = host_status_word();
    if (!p.status) return NVFP4_ERR_CUDA;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.one_over_d = 1.0f / static_cast<float>(p.D);
    // Whole vectors of V values on their boundaries, for V = 8, then 4; else a value per thread.
    const int eb = type_bytes(a->x_type), nb = type_bytes(p.norm_type), cb = p.cache_type == NVFP4_BF16 ? 2 : 1;
    auto fits = [&](int v) {
        auto on = [&](const void* q, int bytes) { return aligned(q, bytes < 16 ? bytes : 16); };
        bool ok = p.D % (2 * v) == 0 && p.D <= 32 * 2 * v && p.half % v == 0 && on(p.q_out, 2 * v) && on(p.q_norm, nb * v) &&
                  on(p.k_norm, nb * v);
        for (int i = 0; i < 3; ++i) ok = ok && on(p.x[i], eb * v) && p.ts[i] % v == 0 && p.hs[i] % v == 0;
        for (int i = 0; i < 2; ++i) ok = ok && on(p.cache[i], cb * v) && p.page_stride[i] % v == 0;  // (E2M1: words of codes)
        return ok;
    };
    const bool f4 = p.cache_type == NVFP4_E2M1;
    const int v = host_variant() == 1 ? 0 : fits(8) ? 8 : fits(4) ? 4 : 0;
    if (v) {
        while ((2 * v << p.lanes_log2) < p.D) ++p.lanes_log2;
        // A token's heads are shared among warps, down to one step each, until the SMs' warps are filled twice
        // (8192 tokens, a warp each: 39.5 us; two warps each: 42.9; four: 44.5).
        const int hpi = 32 >> p.lanes_log2, steps = (p.hq + hpi - 1) / hpi + 2 * ((p.hk + hpi - 1) / hpi);
        const int64_t want = (40ll * host_sm_count() + p.T - 1) / p.T;
        p.shares = static_cast<int>(want < 1 ? 1 : want < steps ? want : steps);
        const int warps = kThreads / 32;
        const int64_t ctas = (static_cast<int64_t>(p.T) * p.shares + warps - 1) / warps;
        const dim3 grid(static_cast<unsigned>(ctas));
        const size_t smem = static_cast<size_t>(warps) * (p.half * sizeof(float2) + (f4 && v == 4 ? 64 * sizeof(uint32_t) : 0));
        const bool f32 = a->x_type == NVFP4_F32;
        if (f4 && v == 4)
            return f32 ? launch(rope_append_kernel<float, 4, true>, grid, dim3(kThreads), smem, st, p)
                       : launch(rope_append_kernel<__nv_bfloat16, 4, true>, grid, dim3(kThreads), smem, st, p);
        if (f4)
            return f32 ? launch(rope_append_kernel<float, 8, true>, grid, dim3(kThreads), smem, st, p)
                       : launch(rope_append_kernel<__nv_bfloat16, 8, true>, grid, dim3(kThreads), smem, st, p);
        if (v == 8)
            return f32 ? launch(rope_append_kernel<float, 8, false>, grid, dim3(kThreads), smem, st, p)
                       : launch(rope_append_kernel<__nv_bfloat16, 8, false>, grid, dim3(kThreads), smem, st, p);
        return f32 ? launch(rope_append_kernel<float, 4, false>, grid, dim3(kThreads), smem, st, p)
                   : launch(rope_append_kernel<__nv_bfloat16, 4, false>, grid, dim3(kThreads), smem, st, p);
    }
    const dim3 grid(p.T, p.hq + 2 * p.hk);
    return a->x_type == NVFP4_F32 ? launch(rope_append_scalar_kernel<float>, grid, dim3(128), p.D * 4, st, p)
                                  : launch(rope_append_scalar_kernel<__nv_bfloat16>, grid, dim3(128), p.D * 4, st, p);
}
