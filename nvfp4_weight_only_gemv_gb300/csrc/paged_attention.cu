// Attention of each sequence's newest tokens over its paged key-value cache.
//
//   s_j = scale * q . k_j  over the keys j that the row sees,   m = max s_j,   l = sum exp(s_j - m)
//   out = sum exp(s_j - m) v_j / l,   lse = m + log l
//
// Keys are taken in one pass: a part of them leaves (m, l, sum exp(s - m) v), and two parts join by
// rescaling both to the larger maximum.

#include "ops_common.cuh"

#include <cuda.h>

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
    // tile kernel
    int* counters;              // workspace: arrivals, two per slot of a part: see kCtasPerSm; zero between calls
    float* part_o;              // workspace: unnormalised sums [2 * grid][rows * group][D]
    float2* part_ml;            // workspace: (m, l) [2 * grid][rows * group]
    int wide_box, tall_box;     // one copy brings all of a block's boxes; all blocks of a tile
    // A kv head's query rows are taken in `chunks` equal chunks of `chunk_rows` (the last may hold fewer),
    // one where a CTA can hold them all; a (kv head, chunk) is a column of a sequence's items.
    int chunks, chunk_rows, columns;
    uint32_t group_inv;         // 2^24 / group, rounded up
    int row_blocks;             // warps of a CTA that share a tile, each with its own query rows
    int page_tiles;             // 16-key blocks per page
    int quad_log2;              // lanes (a power of two) that take a row's 4-value pieces
    uint64_t wait_ns;           // budget of a wait for a copy
    int q_vec;                  // q may be read 8 bytes at a time
};

struct TileParams : AttnParams {
    // k, v: [pages][kv heads][D / 64 pieces of 128 bytes][page][piece] (wide boxes) or
    // [pages][kv heads][1][page][D]; boxes of 16 keys x 128 bytes, or multiples of them
    CUtensorMap map[2];
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
constexpr float kTiny = 1.17549435e-38f;  // 2^-126
constexpr float kSlack = 8.0f; // how far a score may pass the reference maximum, in powers of two
constexpr float kLift = 7.0f;  // powers of two that f16 weights are raised by
constexpr uint64_t kDrainNs = 2000000000ull;
constexpr int kAlignSlack = 3;  // units
constexpr int kMaxGroup = 1024;  // query heads per kv head: 8 group^2 < 2^24, see place_of_row
constexpr int kJoinOnce = 32;  // parts times rows that a thread joins in a single step
// The most CTAs an SM takes in any plan. A CTA has two slots for parts, and a slot two counters: of the item and of
// the group of parts that it is the first of (an item that is cut is the only one to have its first
// part there). So the counters' extent is the device's alone, and every shape finds them at zero.
constexpr int kCtasPerSm = 3;

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

// ------------------------------------------------------------------ tile kernel
//
// One warp takes 16 keys (or a few times 16: TileShape::kKeys) and up to 8 * NT query rows of one
// kv head (rows * group of them) at a time:
//
//   S^T [16 keys x 8 rows]   = K [16 x D] . Q^T        mma m16n8k16, A = keys, B = rows
//   O^T [16 dims x 8 rows]  += V^T [16 x 16 keys] . P^T
//
// Keys stand on the tensor core's 16-row side and the few query rows on its 8-column side, so a
// group of 4 heads wastes half of a column block instead of three quarters of a row block. The
// order of the head's dimensions inside a product is free, so what a lane needs of a key (K) or of
// four keys (V) is whole 16-byte pieces. V's pairs of keys are formed by byte permutes (E4M3 codes
// are widened to f16 behind the permute), P^T by two transposing moves of 8 x 8 halves.
//
// Every warp keeps a ring of its own tiles (kStages of 8 KB at D <= 128) filled by TMA tensor copies
// of 16 keys x 128 bytes, swizzled so that V's pieces are read without a bank conflict and K's with
// two lanes to a bank; K and V of a stage have a barrier each and are requested again as soon as
// they are read, by the warp itself, so no warp waits for another. Straight into registers, with one
// tile a warp in flight, E4M3 with 16 rows reached 4.2 TB/s; by cp.async into the same ring 3.9.
//
// E4M3 keys and values are widened to f16 in registers (exact; mma.sync on E4M3 operands is no
// instruction here but is built from the same conversions and f16 products: it executed 11 % more
// instructions). A query row next to them is f16 too, times a power of two that brings its largest
// magnitude to [2^14, 2^15): exact down to 2^-28 of that, off by 2^-39 of it below.
//
// Probabilities are exp2(s - m) for a reference m that follows the running maximum only when a score
// passes it by more than 2^8: the rescaling of O, and the maximum over the lanes, are then rare.
// Next to bf16 values they enter the products as two bf16 numbers, 16 bits in all: rounded to one,
// the output was 1.35 times as far from 64 bits as fp32's, and the second product costs nothing that
// can be measured (131071 keys: 88.9 us with one, 88.7 with two). The first is rounded down and the
// second kept at 2^-126 or more, so that an infinite value stays infinite; that is as much as exp2's
// flush of smaller weights to zero takes away. Both are zero where the weight is, or a masked key's value
// would reach the row. Next to E4M3 values they are f16, 11 bits against the values' 4, and times 2^7:
// at most 2^15, inside f16's range, and at least 2^7 where a score is the reference, so that a weight is
// off by no more than 2^-32 of the largest where f16's steps of 2^-24 end. (Not raised, the tail behind a key
// 2^26 times as heavy was lost from the sums of the values and not from l.)
//
// The kernel is bound by the cache's bytes.
//
// Work is split over the length without the host knowing the lengths: all (sequence, kv head)
// items lie end to end in units of S tiles (S warps side by side), and every CTA takes an equal
// run of units, or, up to 32 sequences and where that costs little, an equal part of one item
// (3000 keys, 8 kv heads: 32 sequences 65.9 us by parts of items, 33 sequences 67.5 by runs, 0.88 of
// the copy rate both). An item inside one CTA is stored at once; the parts of an item that is cut leave
// (m, l, sum) in the workspace, and the CTA that arrives last joins them in the CTAs' order, so
// the result does not depend on who was last.

template <int DP, int NT, bool F8>
struct TileShape {
    static constexpr int kHalves = F8 ? (DP >= 256 ? 1 : 256 / DP) : (DP >= 128 ? 1 : 128 / DP);  // 16-key blocks
    static constexpr int kKeys = 16 * kHalves;
    static constexpr int kES = F8 ? 1 : 2;                 // bytes per value
    static constexpr int kKC = DP * kES / 64;              // 16-byte chunks of a key row per lane
    static constexpr int kVW = DP * kES / 32;              // 32-bit words of a key's values per lane
    static constexpr int kMT = DP / 16;                    // 16-dim blocks of O
    static constexpr int kQ = DP / 16;                     // operand pairs of a query row block per lane
    static constexpr int kWarps = DP >= 256 ? 8 : 4;
    static constexpr int kCtas = DP >= 256 ? 1 : NT * DP <= 128 ? kCtasPerSm : 2;  // per SM
    static constexpr bool kQRegs = NT * DP <= 256;
    static constexpr int kOStride = DP + 4;                // floats between rows of the merge buffer
    static constexpr int kBoxBytes = DP * kES >= 128 ? 128 : 64;       // of a key in a box
    static constexpr int kBoxes = DP * kES / kBoxBytes;    // boxes of a 16-key block
    static constexpr int kBox = 16 * kBoxBytes;
    static constexpr int kPart = kHalves * kBoxes * kBox;  // K (or V) bytes of a tile
    static constexpr int kStages = DP * kES == 512 ? 1 : NT * DP == 256 ? 3 : NT * DP <= 128 ? 1 : 2;
    static constexpr int kRing = kWarps * kStages * 2 * kPart;
    static constexpr int kMerge = kWarps * 8 * NT * (kOStride * 4 + 8);
    static constexpr int kMain = kRing > kMerge ? kRing : kMerge;  // the merge takes the ring's place
};

__device__ __forceinline__ void barrier_init(uint32_t bar) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void barrier_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool barrier_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n"
                 " mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool barrier_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n"
                 " mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}" : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
__device__ __forceinline__ uint64_t global_ns() {
    uint64_t ns;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(ns));
    return ns;
}
// Waits for a barrier's phase at most `budget` ns (0: polls once); the same answer in every lane.
__device__ __noinline__ bool barrier_wait_slow(uint32_t bar, uint32_t parity, uint64_t budget) {
    const uint64_t begin = global_ns();
    bool ok = false;
    while (!ok && global_ns() - begin <= budget) ok = barrier_try(bar, parity);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ bool barrier_wait(uint32_t bar, uint32_t parity, uint64_t budget) {
    const bool ok = budget == 0 ? barrier_test(bar, parity) : barrier_try(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    return budget != 0 && barrier_wait_slow(bar, parity, budget);
}

// A cache is read once per call and is larger than L2 when it matters: its lines leave L2 first.
__device__ __forceinline__ uint64_t evict_first() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}
__device__ __forceinline__ void copy_box(uint32_t to, const CUtensorMap* map, int x, int key, int head, int page, uint32_t bar,
                                         uint64_t pol) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1, {%2, %3, 0, %4, %5}], [%6], %7;"
        ::"r"(to), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(key), "r"(head), "r"(page), "r"(bar), "l"(pol) : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

template <bool F8>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F8)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

__device__ __forceinline__ uint32_t pack_bf16_down(float lo, float hi) {
    uint32_t d;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The joined weight of a part: 1 where only a NaN sum is left (NaN scores leave m at -inf).
__device__ __forceinline__ float part_weight(float m, float l, float top) {
    return l == 0.0f ? 0.0f : m == -INFINITY ? 1.0f : exp2_fast(m - top);
}

// What a CTA needs of an item: the sequence's length and the keys that its rows see.
struct Span {
    int n, lo, hi_all, lo_all;  // keys [lo, n) for some row, [lo_all, hi_all) for every row
    int units;
};
__device__ __forceinline__ Span span_of(const AttnParams& p, int n, int unit_keys, int align) {
    Span s;
    s.n = n;
    s.hi_all = n - p.rows + 1;
    const int first = p.window > 0 ? s.hi_all - p.window : 0;
    s.lo = first > 0 ? first : 0;
    s.lo_all = p.window > 0 && n > p.window ? n - p.window : 0;
    const int keys = n - (s.lo & ~(align - 1));
    s.units = keys > 0 ? (keys + unit_keys - 1) / unit_keys : 1;  // an empty item still stores its zeros
    return s;
}

// The CTA's run of units, and the part of one item in it. Kept in shared memory: the tile loop
// needs the registers.
struct Run {
    int share, extra;               // units per CTA; the first `extra` CTAs take one more
    int begin, end;                 // this CTA's units
    int seq, head;                  // the item
    int item0, item_end;            // its units
    int first, last;                // the run's part of it
    int cta0, parts, slot0;         // the CTAs that have a part of it: first, how many, the first's slot
    Span span;
};

__device__ __forceinline__ int run_begin(int share, int extra, int cta) { return share * cta + min(cta, extra); }
__device__ __forceinline__ int cta_of(const Run& r, int unit) {
    const int long_units = r.extra * (r.share + 1);
    return unit < long_units ? unit / (r.share + 1) : r.extra + (unit - long_units) / r.share;
}
// The item's CTAs where every CTA takes an equal run. The first one's part is its second segment unless
// its run begins with the item.
__device__ __forceinline__ void find_parts(Run& r) {
    r.cta0 = cta_of(r, r.item0);
    r.parts = cta_of(r, r.item_end - 1) - r.cta0 + 1;
    r.slot0 = 2 * r.cta0 + (run_begin(r.share, r.extra, r.cta0) == r.item0 ? 0 : 1);
}
// Where the run starts: in sequence b, whose heads' units begin at `before`.
__device__ __forceinline__ void enter_run(Run& r, int b, int before, const Span& sp, int cta) {
    r.begin = run_begin(r.share, r.extra, cta);
    r.end = run_begin(r.share, r.extra, cta + 1);
    r.seq = b;
    r.span = sp;
    r.head = (r.begin - before) / sp.units;
    r.item0 = before + r.head * sp.units;
    r.item_end = r.item0 + sp.units;
    r.first = r.begin;
    r.last = min(r.item_end, r.end);
    find_parts(r);
}

// The weights of a row's parts and its totals, for all rows at once: ml[part * step + row] is (m, l) and
// becomes (weight, l), total[row] = (m, l) of the row. Lanes share a row's parts.
__device__ __forceinline__ void weigh_parts(float2* ml, int step, int rows, int count, float2* total) {
    int lanes_log2 = 0;
    while (lanes_log2 < 5 && (1 << lanes_log2) < count) ++lanes_log2;
    const int lanes = 1 << lanes_log2, c0 = threadIdx.x & (lanes - 1), apart = blockDim.x >> lanes_log2;
#pragma unroll 1
    for (int first = 0; first < rows; first += apart) {  // all lanes go through the shuffles
        const int row = first + (threadIdx.x >> lanes_log2);
        const bool in = row < rows;
        float m = -INFINITY, l = 0.0f;
        for (int c = c0; in && c < count; c += lanes) m = fmaxf(m, ml[c * step + row].x);
        for (int o = 1; o < lanes; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        for (int c = c0; in && c < count; c += lanes) {
            const float2 part = ml[c * step + row];
            const float f = part_weight(part.x, part.y, m);
            if (f != 0.0f) l = fmaf(part.y, f, l);
            ml[c * step + row].x = f;
        }
        for (int o = 1; o < lanes; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (in && c0 == 0) total[row] = make_float2(m, l);
    }
}

__device__ __forceinline__ void add_weighed(float4& o, float f, float4 v) {
    const bool on = f != 0.0f;  // else nothing, not even 0 * NaN
    o.x = fmaf(on ? v.x : 0.0f, f, o.x); o.y = fmaf(on ? v.y : 0.0f, f, o.y);
    o.z = fmaf(on ? v.z : 0.0f, f, o.z); o.w = fmaf(on ? v.w : 0.0f, f, o.w);
}
// Four values of a row from its weighed parts, in order.
__device__ __forceinline__ float4 gather(const float2* weight, int step, const char* o, int o_step, int count) {
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int c = 0; c < count; ++c) add_weighed(sum, weight[c * step].x, *reinterpret_cast<const float4*>(o + c * o_step));
    return sum;
}

// The same from parts not weighed yet, one after the other: one trip to shared memory or L2, and
// little code, which counts where every instruction is fetched cold (weighed first, a call with one row
// took 0.7 us longer).
struct Gathered {
    float m = -INFINITY, l = 0.0f;
    float4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    __device__ __forceinline__ void add(float2 ml, float4 v) {
        const float top = fmaxf(m, ml.x);
        const float keep = top == m ? 1.0f : exp2_fast(m - top), f = part_weight(ml.x, ml.y, top);
        m = top;
        l *= keep;
        o.x *= keep; o.y *= keep; o.z *= keep; o.w *= keep;
        if (f == 0.0f) return;
        l = fmaf(ml.y, f, l);
        o.x = fmaf(v.x, f, o.x); o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z); o.w = fmaf(v.w, f, o.w);
    }
};

// Where a row of an item's column goes: the place of (sequence, row, query head) in out and lse; negative
// for the last chunk's padding. Rows (fewer than 8 group) divide by the group through a product, too large by
// row / 2^24 at most, which has to stay below 1 / group: 8 group^2 < 2^24.
__device__ __forceinline__ int64_t place_of_row(const AttnParams& p, int b, int column, int chunk_row) {
    const int h = p.chunks == 1 ? column : column / p.chunks, row = (column - h * p.chunks) * p.chunk_rows + chunk_row;
    if (row >= p.rows * p.group) return -1;
    const int m = static_cast<int>(static_cast<uint32_t>(row) * p.group_inv >> 24), head = h * p.group + row - m * p.group;
    return (static_cast<int64_t>(b) * p.rows + m) * p.hq + head;
}
__device__ __forceinline__ void store_out(const AttnParams& p, int64_t at, int d, float4 o, float l, float vscale) {
    if (at < 0) return;
    const float inv = l == 0.0f ? 0.0f : __fdividef(vscale, l);
    *reinterpret_cast<uint2*>(p.out + at * p.D + d) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
}
__device__ __forceinline__ float log_sum(float2 ml) { return ml.y == 0.0f ? -INFINITY : (ml.x + log2f(ml.y)) * 0.6931471805599453f; }
// lse of all rows of an item's column from their totals.
__device__ __forceinline__ void store_lse(const AttnParams& p, int b, int column, const float2* total) {
    if (!p.lse) return;
#pragma unroll 1
    for (int row = threadIdx.x; row < p.chunk_rows; row += blockDim.x) {
        const int64_t at = place_of_row(p, b, column, row);
        if (at >= 0) p.lse[at] = log_sum(total[row]);
    }
}
__device__ __forceinline__ float value_scale(const AttnParams& p, int column) {
    return p.cache_scale[1] ? p.cache_scale[1][p.chunks == 1 ? column : column / p.chunks] : 1.0f;
}

constexpr int kMaxChunkRows = 128;  // query rows of a CTA in any plan
struct JoinShared {
    float2 ml[kMaxChunkRows];
    int last;
};

// The parts of an item, as slots of the workspace in the CTAs' order.
struct Parts {
    int slot0, cta0;
    __device__ __forceinline__ int slot(int c) const { return c == 0 ? slot0 : 2 * (cta0 + c); }
};

__device__ __forceinline__ int part_bytes(const AttnParams& p) { return p.chunk_rows * (p.D * 4 + 8); }

// How many rows of a part a thread joins, one after the other.
__device__ __forceinline__ int join_turns(const AttnParams& p) {
    const int at_a_time = blockDim.x >> p.quad_log2;
    return (p.chunk_rows + at_a_time - 1) / at_a_time;
}

// Joins parts first, first + step, ... (`count` of them): into the output, or (to >= 0) into the
// workspace slot `to`, which may be the first part's own: a value is read and then replaced by one
// thread, and (m, l) only after all have read them. A thread reads 8 parts of a row at a time; where it
// has several rows, and the parts fit into `room` (the rings' place), they are copied there all at
// once instead, one trip to L2 for all rows. (One row a thread, 32 query heads, us a call and through shared
// memory: 257 keys 8.1 and 8.7, 1024 keys 9.5 both, 131071 keys 84.1 and 85.9; four rows a thread: 25 and 20.)
__device__ __forceinline__ void join_parts(const AttnParams& p, JoinShared& sh, char* room, int room_bytes, const Parts& parts,
                                           int first, int step, int count, int to, int b, int column) {
    const int rows_all = p.chunk_rows, quad = threadIdx.x & ((1 << p.quad_log2) - 1), d = 4 * quad;
    const int o_bytes = rows_all * p.D * 4, ml_bytes = rows_all * 8;
    const bool fits = join_turns(p) > 1 && count * part_bytes(p) <= room_bytes;
    if (fits) {
        const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(room));
#pragma unroll 1
        for (int c = 0; c < count; ++c) {
            const int64_t from = static_cast<int64_t>(parts.slot(first + c * step)) * rows_all;
            const char* const o = reinterpret_cast<const char*>(p.part_o + from * p.D);
            const char* const ml = reinterpret_cast<const char*>(p.part_ml + from);
            for (int i = 16 * threadIdx.x; i < o_bytes; i += 16 * blockDim.x)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + c * o_bytes + i), "l"(o + i) : "memory");
            for (int i = 8 * threadIdx.x; i < ml_bytes; i += 8 * blockDim.x)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at + count * o_bytes + c * ml_bytes + i), "l"(ml + i) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
    }
    const float vscale = value_scale(p, column);
    if (fits) {
        float2* const ml = reinterpret_cast<float2*>(room + count * o_bytes);
        weigh_parts(ml, rows_all, rows_all, count, sh.ml);
        __syncthreads();
#pragma unroll 2
        for (int row = threadIdx.x >> p.quad_log2; row < rows_all; row += blockDim.x >> p.quad_log2) {
            if (d >= p.D) continue;
            const float4 o = gather(ml + row, rows_all, room + (row * p.D + d) * 4, o_bytes, count);
            if (to < 0) store_out(p, place_of_row(p, b, column, row), d, o, sh.ml[row].y, vscale);
            else __stcg(reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(to) * rows_all + row) * p.D + d), o);
        }
    } else {
#pragma unroll 1
        for (int row = threadIdx.x >> p.quad_log2; row < rows_all; row += blockDim.x >> p.quad_log2) {
            if (d >= p.D) continue;
            float* const po = p.part_o + row * p.D + d;
            Gathered a;
#pragma unroll 1
            for (int c = 0; c < count; c += 8) {
                float4 v[8];
                float2 ml[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int from = parts.slot(first + min(c + j, count - 1) * step) * rows_all;
                    ml[j] = __ldcg(p.part_ml + from + row);
                    v[j] = __ldcg(reinterpret_cast<const float4*>(po + static_cast<int64_t>(from) * p.D));
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c + j < count) a.add(ml[j], v[j]);
            }
            if (to < 0) {
                const int64_t at = place_of_row(p, b, column, row);
                store_out(p, at, d, a.o, a.l, vscale);
                if (d == 0 && p.lse && at >= 0) p.lse[at] = log_sum(make_float2(a.m, a.l));
            } else {
                __stcg(reinterpret_cast<float4*>(po + static_cast<int64_t>(to) * rows_all * p.D), a.o);
                if (d == 0) sh.ml[row] = make_float2(a.m, a.l);
            }
        }
        if (to < 0) return;
        __syncthreads();
    }
    if (to < 0) {
        store_lse(p, b, column, sh.ml);
        return;
    }
    __syncthreads();
    for (int row = threadIdx.x; row < rows_all; row += blockDim.x) __stcg(p.part_ml + to * rows_all + row, sh.ml[row]);
}

// The same for parts that do not fit into `room` at once, where a thread has more than 4 rows: as many rows
// of all parts as do fit, turn by turn. us a call, read and this way: 64 rows of 128 values (16 a thread),
// 300 keys 47.8 and 34.8, 20000 keys 84 and 79; E4M3, rows of 256 values 50.8 and 35.8, 121 and 106. With
// two rows a thread it is slower: 1200 keys 12.6 and 14.4. Out of line: inside the common join it cost an E4M3 batch 2.5 %.
__device__ __noinline__ void join_in_turns(const AttnParams& p, JoinShared& sh, char* room, int room_bytes, const Parts& parts,
                                           int first, int step, int count, int to, int b, int column) {
    const int rows_all = p.chunk_rows, quad = threadIdx.x & ((1 << p.quad_log2) - 1), d = 4 * quad;
    const float vscale = value_scale(p, column);
    const int fit = room_bytes / (count * (p.D * 4 + 8)), turns = (rows_all + fit - 1) / fit, most = (rows_all + turns - 1) / turns;
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(room));
#pragma unroll 1
    for (int row0 = 0; row0 < rows_all; row0 += most) {
        const int rows = min(most, rows_all - row0), o_bytes = rows * p.D * 4, ml_bytes = rows * 8;
#pragma unroll 1
        for (int c = 0; c < count; ++c) {
            const int64_t from = static_cast<int64_t>(parts.slot(first + c * step)) * rows_all + row0;
            const char* const o = reinterpret_cast<const char*>(p.part_o + from * p.D);
            const char* const ml = reinterpret_cast<const char*>(p.part_ml + from);
            for (int i = 16 * threadIdx.x; i < o_bytes; i += 16 * blockDim.x)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at + c * o_bytes + i), "l"(o + i) : "memory");
            for (int i = 8 * threadIdx.x; i < ml_bytes; i += 8 * blockDim.x)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at + count * o_bytes + c * ml_bytes + i), "l"(ml + i) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncthreads();
        float2* const ml = reinterpret_cast<float2*>(room + count * o_bytes);
        weigh_parts(ml, rows, rows, count, sh.ml + row0);
        __syncthreads();
#pragma unroll 2
        for (int row = threadIdx.x >> p.quad_log2; row < rows; row += blockDim.x >> p.quad_log2) {
            if (d >= p.D) continue;
            const float4 o = gather(ml + row, rows, room + (row * p.D + d) * 4, o_bytes, count);
            if (to < 0) store_out(p, place_of_row(p, b, column, row0 + row), d, o, sh.ml[row0 + row].y, vscale);
            else __stcg(reinterpret_cast<float4*>(p.part_o + (static_cast<int64_t>(to) * rows_all + row0 + row) * p.D + d), o);
        }
        if (row0 + most < rows_all) __syncthreads();
    }
    if (to < 0) {
        store_lse(p, b, column, sh.ml);
        return;
    }
    for (int row = threadIdx.x; row < rows_all; row += blockDim.x) __stcg(p.part_ml + to * rows_all + row, sh.ml[row]);
}

// True in the CTA that is the last of `of` to come by `counter`, which it leaves at zero. The CTA's
// stores come before its arrival, and the other CTAs' before what the last one reads.
__device__ __forceinline__ bool arrive_last(JoinShared& sh, int* counter, int of) {
    __syncthreads();
    if (threadIdx.x == 0) {
        int old;
        asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
        sh.last = old == of - 1;
        if (sh.last) *counter = 0;
    }
    __syncthreads();
    return sh.last != 0;
}

// Called by every CTA that has left a part of an item in the workspace: the last of them joins the
// parts. Many parts meet in two steps, first groups of neighbours (by the last of each), then the
// groups. Out of line, so that its registers are not the tile loop's.
__device__ __noinline__ void finish_item(const AttnParams& p, JoinShared& sh, const Run& r, char* room, int room_bytes) {
    const int cta0 = r.cta0, parts = r.parts;
    const Parts at{r.slot0, cta0};
    int* const done = p.counters + 2 * at.slot(0);
    int size = parts;
    auto join = [&](int first, int step, int count, int to) {
        const int a_row = count * (p.D * 4 + 8);
        if (join_turns(p) > 4 && p.chunk_rows * a_row > room_bytes && a_row <= room_bytes)
            join_in_turns(p, sh, room, room_bytes, at, first, step, count, to, r.seq, r.head);
        else
            join_parts(p, sh, room, room_bytes, at, first, step, count, to, r.seq, r.head);
    };
    if (parts > 4 && parts * join_turns(p) > kJoinOnce && (join_turns(p) == 1 || parts * part_bytes(p) > room_bytes)) {
        size = 3;
        while (size * size < parts) ++size;
        const int first = (static_cast<int>(blockIdx.x) - cta0) / size * size, count = min(size, parts - first);
        if (!arrive_last(sh, p.counters + 2 * at.slot(first) + 1, count)) return;
        join(first, 1, count, at.slot(first));
    }
    const int groups = (parts + size - 1) / size, of = size < parts ? groups : parts;
    if (arrive_last(sh, done, of)) join(0, size < parts ? size : 1, of, -1);
}

template <int DP, int NT, bool F8>
__global__ void __launch_bounds__(TileShape<DP, NT, F8>::kWarps * 32, TileShape<DP, NT, F8>::kCtas)
paged_attention_tile_kernel(const __grid_constant__ TileParams p) {
    using T = TileShape<DP, NT, F8>;
    constexpr int H = T::kHalves, W = T::kWarps, kThreads = W * 32;
    constexpr int kRowsW = 8 * NT;
    constexpr float lift = F8 ? kLift : 0.0f;
    extern __shared__ uint8_t smem_raw[];
    // rings [W][kStages][K, V], on a boundary of the swizzle's pattern; then s_q
    float* const smem = reinterpret_cast<float*>(smem_raw + (-static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)) & 1023u));
    __shared__ __align__(8) uint64_t s_bar[W][T::kStages][2];
    __shared__ int s_scan[W];
    __shared__ float s_f[8 * NT * W];  // rows' factors (not kQRegs)
    __shared__ Run s_run;
    __shared__ JoinShared s_join;
    float* s_o = smem;                                        // merge, in the rings' place: [W][kRowsW][kOStride]
    float2* s_ml = reinterpret_cast<float2*>(s_o + W * kRowsW * T::kOStride);  // [W][kRowsW]
    uint2* s_q = reinterpret_cast<uint2*>(smem + T::kMain / 4);  // [row_blocks][NT][kQ][32] (not kQRegs)

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int rb = warp % p.row_blocks, stream = warp / p.row_blocks, streams = W / p.row_blocks;
    const int rows_all = p.rows * p.group;
    const int unit_keys = streams * T::kKeys, align = p.tall_box ? T::kKeys : 16;

    pdl_launch_dependents();
    const uint32_t bars = static_cast<uint32_t>(__cvta_generic_to_shared(&s_bar[warp][0][0]));
    if (lane < 2 * T::kStages) barrier_init(bars + 8 * lane);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (tid < 2) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&p.map[tid])) : "memory");
    pdl_wait();

    // --- the CTA's part of the work. All (sequence, kv head) items lie end to end in units; a CTA takes
    // an equal run of them, or, where that costs little, an equal part of a single item, which
    // saves it a second start and a second join (worth about kAlignSlack units).
    Run run;
    const int cta = blockIdx.x, grid = gridDim.x;
    if (p.seqs <= 32) {
        // every warp for itself, a sequence per lane
        Span sp{};
        if (lane < p.seqs) sp = span_of(p, length_of(p, lane), unit_keys, align);
        auto prefix = [&](int v) {  // inclusive
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int w = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += w;
            }
            return v;
        };
        const int incl = prefix(sp.units), total = __shfl_sync(0xffffffffu, incl, 31) * p.columns;
        // An item of few units is not split where a join takes longer than they do. us split and not: 2
        // units of one row 8.8 and 7.0, 5 units of one row 8.7 and 9.8, of two 11.1 and 12.0, of four
        // 13.3 and 12.5, of eight 21.8 and 20.2 (rows that a thread joins).
        const int least = (total + grid - 1) / grid, alone = min(2 + join_turns(p), 6);
        int n = 0, before = 0;  // CTAs of an item of this lane's sequence; CTAs or units before the sequence
        bool whole_items = false;
        for (int load = least; load <= least + kAlignSlack && !whole_items; ++load) {
            n = sp.units <= alone ? sp.units > 0 : (sp.units + load - 1) / load;
            whole_items = __reduce_add_sync(0xffffffffu, n) * p.columns <= grid;
        }
        bool here;
        if (whole_items) {
            before = (prefix(n) - n) * p.columns;
            here = cta >= before && cta < before + n * p.columns;
        } else {
            run.share = total / grid;  // more units than CTAs, or a unit per CTA would have done
            run.extra = total - run.share * grid;
            before = (incl - sp.units) * p.columns;
            const int begin = run_begin(run.share, run.extra, cta);
            here = begin >= before && begin < before + sp.units * p.columns;
        }
        const uint32_t owner = __ballot_sync(0xffffffffu, here);
        if (owner == 0) return;
        const int b = __ffs(owner) - 1;
        n = __shfl_sync(0xffffffffu, n, b);
        before = __shfl_sync(0xffffffffu, before, b);
        Span at;
        at.n = __shfl_sync(0xffffffffu, sp.n, b);
        at.lo = __shfl_sync(0xffffffffu, sp.lo, b);
        at.hi_all = __shfl_sync(0xffffffffu, sp.hi_all, b);
        at.lo_all = __shfl_sync(0xffffffffu, sp.lo_all, b);
        at.units = __shfl_sync(0xffffffffu, sp.units, b);
        if (whole_items) {
            run.seq = b;
            run.span = at;
            run.head = (cta - before) / n;
            run.cta0 = before + run.head * n;
            run.parts = n;
            run.slot0 = 2 * run.cta0;
            const int part = cta - run.cta0, even = at.units / n, odd = at.units - even * n;
            run.item0 = 0;
            run.item_end = at.units;
            run.begin = run.first = run_begin(even, odd, part);
            run.end = run.last = run_begin(even, odd, part + 1);
        } else {
            enter_run(run, b, before, at, cta);
        }
        if (tid == 0) s_run = run;
    } else {
        const int per = (p.seqs + kThreads - 1) / kThreads;
        int mine = 0;
        for (int i = 0; i < per; ++i) {
            const int b = tid * per + i;
            if (b < p.seqs) mine += span_of(p, length_of(p, b), unit_keys, align).units;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) s_scan[warp] = incl;
        __syncthreads();
        int total = 0, before = incl - mine;
        for (int i = 0; i < W; ++i) {
            if (i < warp) before += s_scan[i];
            total += s_scan[i];
        }
        total *= p.columns;
        const int ctas = min(total, grid);
        if (cta >= ctas) return;
        run.share = total / ctas;
        run.extra = total - run.share * ctas;
        const int begin = run_begin(run.share, run.extra, cta);
        before *= p.columns;
        if (begin >= before && begin < before + mine * p.columns) {
            int b = tid * per;
            Span sp;
            for (;; ++b) {
                sp = span_of(p, length_of(p, b), unit_keys, align);
                if (begin < before + sp.units * p.columns) break;
                before += sp.units * p.columns;
            }
            enter_run(run, b, before, sp, cta);
            s_run = run;
        }
        __syncthreads();
        run = s_run;
    }

    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + warp * (T::kStages * 2 * T::kPart);
    uint32_t cur = 0;      // the stage of the tile in work
    uint32_t parity = 0;   // of the phase that the stage in work completes; the stages take turns
    bool dead = false;     // a copy did not come in time
    // offsets of this lane's pieces in a box: K's of rows g (and g + 8), V's of rows 2t and 2t + 1
    // (and 8 further). A 16-byte piece j of row r stands at piece j ^ (r & 7), in rows of 64 bytes at
    // j ^ (r >> 1 & 3).
    constexpr int kRow = T::kBoxBytes;
    const uint32_t k_off = kRow == 128 ? g * 128 + ((t ^ g) << 4) : g * 64 + ((t ^ (g >> 1 & 3)) << 4);
    auto v_piece = [&](int r) -> uint32_t {
        return kRow == 128 ? r * 128 + ((g ^ r) << 4) : r * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
    };
    const uint32_t v_off[2] = {v_piece(2 * t), v_piece(2 * t + 1)};

    // --- the ring's state. Tiles of this warp: stream, stream + streams, ... of the run's part of an item. A
    // tile's first 16-key block stands at block `slot` of the sequence's page `page`; both walk along.
    Span sp;
    int h, base;                    // the item's kv head, the first tile's first key
    const int32_t* pages;
    int tile, tile_end;
    const int step_page = streams * H / p.page_tiles, step_slot = streams * H % p.page_tiles;
    int next_page = 0, next_slot = 0;
    int id[H], next_id[H];          // page ids of the requested tile, and of the one after it
    int at[H], next_at[H];          // the block's first key in its page
    uint32_t bad = 0, bads = 0;     // blocks whose page id is out of range: requested tile; tiles in the ring

    // looks up the tile after the requested one
    auto look_up = [&](int tl) {
        int pg = next_page, sl = next_slot;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            if (i > 0 && p.tall_box) break;
            next_id[i] = 0;
            if (tl < tile_end && base + tl * T::kKeys + 16 * i < sp.n) next_id[i] = pages[pg];
            next_at[i] = 16 * sl;
            if (++sl == p.page_tiles) { sl = 0; ++pg; }
        }
        next_slot += step_slot;
        next_page += step_page;
        if (next_slot >= p.page_tiles) { next_slot -= p.page_tiles; ++next_page; }
    };
    auto take = [&]() {
        bad = 0;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            if (i > 0 && p.tall_box) break;
            id[i] = next_id[i];
            at[i] = next_at[i];
            if (static_cast<unsigned>(id[i]) >= static_cast<unsigned>(p.pages)) {
                if (lane == 0) atomicOr(&g_attention_status, NVFP4_DEV_BAD_PAGE);
                id[i] = 0;
                bad |= p.tall_box ? (1u << H) - 1 : 1u << i;
            }
        }
    };
    // copies K (which = 0) or V of the taken tile to a stage; every lane is through with its last use
    auto request = [&](uint32_t stage, int which) {
        __syncwarp();
        const uint32_t bar = bars + 16 * stage + 8 * which, to = ring + (2 * stage + which) * T::kPart;
        if (lane == 0) {
            const uint64_t pol = evict_first();
            barrier_expect(bar, T::kPart);
#pragma unroll
            for (int i = 0; i < H; ++i)
#pragma unroll
                for (int x = 0; x < T::kBoxes; ++x)
                    if ((i == 0 || !p.tall_box) && (x == 0 || !p.wide_box))
                        copy_box(to + (i * T::kBoxes + x) * T::kBox, &p.map[which], x * (T::kBoxBytes / T::kES), at[i], h, id[i], bar, pol);
        }
    };
    auto enter_item = [&]() {
        sp = run.span;
        h = p.chunks == 1 ? run.head : run.head / p.chunks;
        // whole tiles stand in one page where pages are multiples of a tile
        base = sp.lo & ~(p.tall_box ? T::kKeys - 1 : 15);
        pages = p.table + run.seq * p.table_stride;
        tile_end = (run.last - run.item0) * streams;
        tile = (run.first - run.item0) * streams + stream;
        next_page = ((base >> 4) + tile * H) / p.page_tiles;
        next_slot = ((base >> 4) + tile * H) % p.page_tiles;
        bads = 0;
        look_up(tile);
    };
    auto fill_ring = [&]() {
#pragma unroll
        for (int st = 0; st < T::kStages; ++st) {
            const int tl = tile + st * streams;
            if (tl < tile_end && !dead) {
                take();
                const uint32_t stage = cur + st < T::kStages ? cur + st : cur + st - T::kStages;
                request(stage, 0);
                request(stage, 1);
                bads |= bad << 8 * st;
                look_up(tl + streams);
            }
        }
    };

    for (;;) {
        const int b = run.seq;
        enter_item();
        const int row0 = (run.head - h * p.chunks) * p.chunk_rows + rb * kRowsW;  // this warp's first query row
        const int rows_end = min(rows_all, (run.head - h * p.chunks + 1) * p.chunk_rows);
        const float kscale = p.cache_scale[0] ? p.cache_scale[0][h] : 1.0f;
        int k_taken = 0;                // the wait that failed was for V: this tile's K had come
        auto arrived = [&](int which) { return barrier_wait(bars + 16 * cur + 8 * which, parity, p.wait_ns); };
        // every key of the tile is there for every row
        auto whole = [&](int tl) {
            const int key = base + tl * T::kKeys;
            return key >= sp.lo_all && key + T::kKeys <= sp.hi_all;
        };

        // --- query rows as the scores' B operand
        auto load_q = [&](int nt, uint2 (&raw)[T::kQ]) {
            const int row = row0 + 8 * nt + g, m = static_cast<int>(static_cast<uint32_t>(row) * p.group_inv >> 24);
            const __nv_bfloat16* q = p.q + (static_cast<int64_t>(b) * p.rows + m) * p.q_ts +
                                     static_cast<int64_t>(h * p.group + row - m * p.group) * p.q_hs;
            const bool live = row < rows_end;
#pragma unroll
            for (int i = 0; i < T::kQ; ++i) {  // 4 values each, in the order of the keys' registers
                const int d = F8 ? 16 * (t + 4 * (i >> 2)) + 4 * (i & 3) : 8 * (t + 4 * (i >> 1)) + 4 * (i & 1);
                raw[i] = make_uint2(0, 0);
                if (live && d < p.D) {
                    if (p.q_vec) {
                        raw[i] = *reinterpret_cast<const uint2*>(q + d);
                    } else {
                        const uint16_t* w = reinterpret_cast<const uint16_t*>(q + d);
                        raw[i] = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
                    }
                }
            }
        };
        // The factor from scores to base-2 units is made positive (its sign goes to q), so that the maximum
        // can be taken over raw scores; a zero becomes 2^-126, or masked scores would be NaN.
        auto convert_q = [&](uint2 (&raw)[T::kQ]) {
            float f = p.scale * 1.4426950408889634f * kscale;
            const uint32_t flip = f < 0.0f ? 0x80008000u : 0u;
            f = fabsf(f);
            if constexpr (F8) {
                uint32_t tops = 0;  // magnitudes, two a word
#pragma unroll
                for (int i = 0; i < T::kQ; ++i) tops = __vmaxu2(__vmaxu2(tops, raw[i].x & 0x7fff7fffu), raw[i].y & 0x7fff7fffu);
                uint32_t top = max(tops & 0xffffu, tops >> 16);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // (an infinity's exponent leaves the finite values next to it below 2^15 too)
                const int up = top == 0 ? 0 : min(14 - (static_cast<int>(top >> 7) - 127), 126);
                const float mul = __int_as_float((127 + up) << 23);
                f *= __int_as_float((127 - up) << 23);
                auto narrow = [&](uint32_t w) { return pack_f16(bf16_lo(w) * mul, bf16_hi(w) * mul); };
#pragma unroll
                for (int i = 0; i < T::kQ; ++i) raw[i] = make_uint2(narrow(raw[i].x), narrow(raw[i].y));
            }
#pragma unroll
            for (int i = 0; i < T::kQ; ++i) raw[i] = make_uint2(raw[i].x ^ flip, raw[i].y ^ flip);
            return f < 1.1754943508e-38f ? 1.1754943508e-38f : f;
        };
        uint2 qf[T::kQRegs ? NT : 1][T::kQ];
        float zf[NT][2];  // what turns a score into base-2 units, for rows 2t, 2t + 1 of each block
        if constexpr (T::kQRegs) {  // on their way while the first tiles are requested
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) load_q(nt, qf[nt]);
        }
        fill_ring();
        if constexpr (T::kQRegs) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float f = convert_q(qf[nt]);
                zf[nt][0] = F8 ? __shfl_sync(0xffffffffu, f, 8 * t) : f;
                zf[nt][1] = F8 ? __shfl_sync(0xffffffffu, f, 8 * t + 4) : f;
            }
        } else {  // the warps that share the rows share the work
#pragma unroll 1
            for (int nt = stream; nt < NT; nt += streams) {
                load_q(nt, qf[0]);
                const float f = convert_q(qf[0]);
                if (t == 0) s_f[(rb * NT + nt) * 8 + g] = f;
#pragma unroll
                for (int i = 0; i < T::kQ; ++i) s_q[((rb * NT + nt) * T::kQ + i) * 32 + lane] = qf[0][i];
            }
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                zf[nt][0] = s_f[(rb * NT + nt) * 8 + 2 * t];
                zf[nt][1] = s_f[(rb * NT + nt) * 8 + 2 * t + 1];
            }
        }
        auto query = [&](int nt, int i) {
            if constexpr (T::kQRegs) return qf[nt][i];
            else return s_q[((rb * NT + nt) * T::kQ + i) * 32 + lane];
        };

        float o[NT][T::kMT][4], mx[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = mx[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
#pragma unroll
            for (int mt = 0; mt < T::kMT; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.0f;
        }

        const bool was_dead = dead;
        for (; tile < tile_end && !dead; tile += streams) {
            // --- scores
            if (!arrived(0)) { dead = true; break; }
            const uint32_t kt = ring + 2 * cur * T::kPart + k_off, vt = ring + (2 * cur + 1) * T::kPart;
            float s[H][NT][4];
            float s2[H][NT][4];  // a second chain of sums where there would be one
            constexpr bool kTwo = H * NT == 1;
#pragma unroll
            for (int i = 0; i < H; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][nt][e] = s2[i][nt][e] = 0.0f;
#pragma unroll
            for (int c = 0; c < T::kKC; ++c) {
                uint4 x[H], y[H];
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    // piece t + 4c of rows g and g + 8
                    const uint32_t from = (kt ^ (kRow == 128 ? 64 * (c & 1) : 0)) + (i * T::kBoxes + (kRow == 128 ? c >> 1 : c)) * T::kBox;
                    x[i] = lds16(from);
                    y[i] = lds16(from + 8 * kRow);
                }
                if constexpr (F8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t a[H][4];
#pragma unroll
                        for (int i = 0; i < H; ++i) {
                            const uint32_t xw = e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w;
                            const uint32_t yw = e == 0 ? y[i].x : e == 1 ? y[i].y : e == 2 ? y[i].z : y[i].w;
                            a[i][0] = e4m3x2_f16x2(xw); a[i][2] = e4m3x2_f16x2(xw >> 16);
                            a[i][1] = e4m3x2_f16x2(yw); a[i][3] = e4m3x2_f16x2(yw >> 16);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 q = query(nt, 4 * c + e);
#pragma unroll
                            for (int i = 0; i < H; ++i)
                                mma<true>(kTwo && (e & 1) ? s2[i][nt] : s[i][nt], a[i][0], a[i][1], a[i][2], a[i][3], q.x, q.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 q = query(nt, 2 * c + e);
#pragma unroll
                            for (int i = 0; i < H; ++i)
                                mma<false>(kTwo && e ? s2[i][nt] : s[i][nt], e ? x[i].z : x[i].x, e ? y[i].z : y[i].x,
                                           e ? x[i].w : x[i].y, e ? y[i].w : y[i].y, q.x, q.y);
                        }
                }
            }
            if constexpr (kTwo) {
#pragma unroll
                for (int e = 0; e < 4; ++e) s[0][0][e] += s2[0][0][e];
            }
            const uint32_t bad_now = bads & 0xffu;
            const bool edge = !whole(tile) || bad_now != 0;
            const int next = tile + T::kStages * streams;
            bads >>= 8;
            if (next < tile_end) {
                take();
                request(cur, 0);
                bads |= bad << 8 * (T::kStages - 1);
            }
            // --- mask, reference maximum, probabilities
            if (edge) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int row = row0 + 8 * nt + 2 * t + c;
                        const int hi = row < rows_end ? sp.hi_all + row / p.group : 0, lo = p.window > 0 ? hi - p.window : 0;
#pragma unroll
                        for (int i = 0; i < H; ++i)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                const int key = base + tile * T::kKeys + 16 * i + 8 * r + g;
                                if (key < lo || key >= hi || (bad_now >> i & 1u)) s[i][nt][2 * r + c] = -INFINITY;
                            }
                    }
            }
            float top[NT][2];
            bool passed = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float z = -INFINITY;
#pragma unroll
                    for (int i = 0; i < H; ++i) z = fmaxf(z, fmaxf(s[i][nt][c], s[i][nt][2 + c]));
                    top[nt][c] = z * zf[nt][c];
                    passed |= top[nt][c] > mx[nt][c] + kSlack;
                }
            if (__any_sync(0xffffffffu, passed)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float keep[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float z = top[nt][c];
                        z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 4));
                        z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 8));
                        z = fmaxf(fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 16)), mx[nt][c]);
                        keep[c] = z == mx[nt][c] ? 1.0f : exp2_fast(mx[nt][c] - z);
                        mx[nt][c] = z;
                        l[nt][c] *= keep[c];
                    }
#pragma unroll
                    for (int mt = 0; mt < T::kMT; ++mt) {
                        o[nt][mt][0] *= keep[0]; o[nt][mt][2] *= keep[0];
                        o[nt][mt][1] *= keep[1]; o[nt][mt][3] *= keep[1];
                    }
                }
            }
            uint32_t pb[H][NT][2], pl[H][NT][2];  // weights; bf16: their first and last 8 bits
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float m0 = (mx[nt][0] == -INFINITY ? 0.0f : mx[nt][0]) - lift, m1 = (mx[nt][1] == -INFINITY ? 0.0f : mx[nt][1]) - lift;
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    float e[4];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        e[2 * r] = exp2_fast(fmaf(s[i][nt][2 * r], zf[nt][0], -m0));
                        e[2 * r + 1] = exp2_fast(fmaf(s[i][nt][2 * r + 1], zf[nt][1], -m1));
                        l[nt][0] += e[2 * r];
                        l[nt][1] += e[2 * r + 1];
                        if constexpr (F8) {
                            pb[i][nt][r] = transpose8x8(pack_f16(e[2 * r], e[2 * r + 1]));
                        } else {
                            const uint32_t word = pack_bf16_down(e[2 * r], e[2 * r + 1]);
                            pb[i][nt][r] = transpose8x8(word);
                            // weights are zero or 2^-126 and more
                            pl[i][nt][r] = transpose8x8(pack_bf16(fmaxf(e[2 * r] - bf16_lo(word), fminf(e[2 * r], kTiny)),
                                                                  fmaxf(e[2 * r + 1] - bf16_hi(word), fminf(e[2 * r + 1], kTiny))));
                        }
                    }
                }
            }
            // --- O^T += V^T P^T. A weight of zero must also silence what is not finite: in tiles that
            // some row sees only in part, such values are taken row by row of the sequence below.
            if (!arrived(1)) { dead = true; k_taken = 1; break; }
            uint32_t vr[4][T::kVW];
            auto load_v = [&](int i) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // keys 2t, 2t + 1, 2t + 8, 2t + 9
                    const uint32_t from = vt + i * (T::kBoxes * T::kBox) + v_off[k & 1] + (k >> 1) * (8 * kRow);
                    if constexpr (T::kVW == 2) {
                        const uint2 v = lds8(from);
                        vr[k][0] = v.x; vr[k][1] = v.y;
                    } else {
#pragma unroll
                        for (int c = 0; c < T::kVW / 4; ++c) {
                            const uint4 v = lds16(from + c * T::kBox);
                            vr[k][4 * c] = v.x; vr[k][4 * c + 1] = v.y; vr[k][4 * c + 2] = v.z; vr[k][4 * c + 3] = v.w;
                        }
                    }
                }
            };
            // keeps values of keys [lo, hi) of block i (of none if its page is bad), zeros the others
            auto keep_v = [&](int i, int lo, int hi) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int key = base + tile * T::kKeys + 16 * i + 2 * t + (k & 1) + 8 * (k >> 1);
                    if (key < lo || key >= hi || (bad_now >> i & 1u)) {
#pragma unroll
                        for (int w = 0; w < T::kVW; ++w) vr[k][w] = 0;
                    }
                }
            };
            auto operands = [&](int mt, uint32_t (&a)[4]) {
                if constexpr (F8) {
                    const int w = mt >> 1;
                    const uint32_t sel = mt & 1 ? 0x7362u : 0x5140u;
                    const uint32_t x = __byte_perm(vr[0][w], vr[1][w], sel), y = __byte_perm(vr[2][w], vr[3][w], sel);
                    a[0] = e4m3x2_f16x2(x); a[1] = e4m3x2_f16x2(x >> 16);
                    a[2] = e4m3x2_f16x2(y); a[3] = e4m3x2_f16x2(y >> 16);
                } else {
                    a[0] = __byte_perm(vr[0][mt], vr[1][mt], 0x5410); a[1] = __byte_perm(vr[0][mt], vr[1][mt], 0x7632);
                    a[2] = __byte_perm(vr[2][mt], vr[3][mt], 0x5410); a[3] = __byte_perm(vr[2][mt], vr[3][mt], 0x7632);
                }
            };
            bool special = false;
            if (edge && (p.rows > 1 || p.window > 0)) {
#pragma unroll 1
                for (int i = 0; i < H; ++i) {
                    load_v(i);
                    keep_v(i, sp.lo, sp.n);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int w = 0; w < T::kVW; ++w) {
                            const uint32_t x = vr[k][w];
                            if constexpr (F8) special |= (((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                            else special |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
                        }
                }
                special = __any_sync(0xffffffffu, special);
            }
            if (!special) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    load_v(i);
                    if (edge) keep_v(i, sp.lo, sp.n);  // what a page holds beyond the sequence may be anything
#pragma unroll
                    for (int mt = 0; mt < T::kMT; ++mt) {
                        uint32_t a[4];
                        operands(mt, a);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma<F8>(o[nt][mt], a[0], a[1], a[2], a[3], pb[i][nt][0], pb[i][nt][1]);
                            if constexpr (!F8) mma<F8>(o[nt][mt], a[0], a[1], a[2], a[3], pl[i][nt][0], pl[i][nt][1]);
                        }
                    }
                }
            } else {
#pragma unroll 1
                for (int m = 0; m < p.rows; ++m) {
                    const int hi = sp.hi_all + m, lo = p.window > 0 ? hi - p.window : 0;
#pragma unroll
                    for (int i = 0; i < H; ++i) {
                        load_v(i);
                        keep_v(i, max(lo, 0), min(hi, sp.n));
#pragma unroll
                        for (int mt = 0; mt < T::kMT; ++mt) {
                            uint32_t a[4];
                            operands(mt, a);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                mma<F8>(d, a[0], a[1], a[2], a[3], pb[i][nt][0], pb[i][nt][1]);
                                if constexpr (!F8) mma<F8>(d, a[0], a[1], a[2], a[3], pl[i][nt][0], pl[i][nt][1]);
                                const int row = row0 + 8 * nt + 2 * t;
                                if (row / p.group == m) { o[nt][mt][0] += d[0]; o[nt][mt][2] += d[2]; }
                                if ((row + 1) / p.group == m) { o[nt][mt][1] += d[1]; o[nt][mt][3] += d[3]; }
                            }
                        }
                    }
                }
            }
            if (next < tile_end) {
                request(cur, 1);
                look_up(next + streams);
            }
            if (++cur == T::kStages) { cur = 0; parity ^= 1; }
        }
        if (dead && !was_dead) {
            // the result is unspecified, but no copy may outlive the CTA: what was requested and has not
            // been waited for is K of this tile or of the one after the ring's, and all the ring's V
            if (lane == 0) atomicOr(&g_attention_status, NVFP4_DEV_TIMEOUT);
#pragma unroll 1
            for (int st = 0; st < 2 * T::kStages; ++st) {
                const int ahead = (st >> 1) + (st & 1 ? 0 : k_taken);  // tiles after this one
                const uint32_t turn = cur + ahead, stage = turn % T::kStages;
                if (tile + ahead * streams < tile_end)
                    barrier_wait(bars + 16 * stage + 8 * (st & 1), parity ^ (turn / T::kStages & 1), kDrainNs);
            }
            tile = tile_end;
        }
        __syncthreads();  // every warp is through with its ring

        // --- the warps' parts meet in shared memory
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float v = l[nt][c];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int r = 8 * nt + 2 * t + c;
                if (g == 0) s_ml[warp * kRowsW + r] = make_float2(mx[nt][c] - lift, v);  // what l and o refer to
#pragma unroll
                for (int x = 0; x < T::kMT / 2; ++x) {
                    const int d = !F8 ? 64 * (x >> 1) + 8 * g + 4 * (x & 1) : DP == 64 ? 8 * g + 4 * x : 128 * (x >> 2) + 16 * g + 4 * (x & 3);
                    *reinterpret_cast<float4*>(s_o + (warp * kRowsW + r) * T::kOStride + d) =
                        make_float4(o[nt][2 * x][c], o[nt][2 * x][2 + c], o[nt][2 * x + 1][c], o[nt][2 * x + 1][2 + c]);
                }
            }
        __syncthreads();
        const Run r = s_run;
        const bool direct = r.parts == 1;
        const float vscale = value_scale(p, r.head);
        const int apart = p.row_blocks * kRowsW;
        const int64_t slot_row = (2 * static_cast<int64_t>(blockIdx.x) + (r.first == r.begin ? 0 : 1)) * p.chunk_rows;
        const int d = 4 * (tid & ((1 << p.quad_log2) - 1)), row1 = tid >> p.quad_log2;
#pragma unroll 1
        for (int row = row1; row < p.chunk_rows; row += kThreads >> p.quad_log2) {
            if (d >= p.D) break;
            const float4* const o = reinterpret_cast<const float4*>(s_o + row * T::kOStride + d);
            Gathered a;
#pragma unroll 1
            for (int st = 0; st < streams; ++st) a.add(s_ml[st * apart + row], o[st * apart * (T::kOStride / 4)]);
            if (direct) {
                const int64_t at = place_of_row(p, r.seq, r.head, row);
                store_out(p, at, d, a.o, a.l, vscale);
                if (d == 0 && p.lse && at >= 0) p.lse[at] = log_sum(make_float2(a.m, a.l));
            } else {
                __stcg(reinterpret_cast<float4*>(p.part_o + (slot_row + row) * p.D + d), a.o);
                if (d == 0) __stcg(p.part_ml + slot_row + row, make_float2(a.m, a.l));
            }
        }
        if (!direct) finish_item(p, s_join, s_run, reinterpret_cast<char*>(smem), T::kMain);
        if (r.last == r.end) return;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the merge buffer is the rings' again
        __syncthreads();  // and s_run and s_q are free
        if (tid == 0) {
            Run& n = s_run;
            if (++n.head == p.columns) {
                n.head = 0;
                ++n.seq;
                n.span = span_of(p, length_of(p, n.seq), unit_keys, align);
            }
            n.first = n.item0 = r.item_end;
            n.item_end = n.item0 + n.span.units;
            n.last = min(n.item_end, n.end);
            find_parts(n);
        }
        __syncthreads();
        run = s_run;
    }
}

cudaError_t read_status(int* bits) {
    const int zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, g_attention_status, sizeof(int));
    return e != cudaSuccess || *bits == 0 ? e : cudaMemcpyToSymbol(g_attention_status, &zero, sizeof(int));
}
const bool g_registered = register_status(read_status);

// The tile kernel's instance for a head size and number of query rows per kv head: the head is
// padded to 64, 128 or 256 in registers, rows to blocks of 8 NT times the warps that share a tile.
struct TilePlan {
    int dp = 0, nt = 1, row_blocks = 1, ctas_per_sm = 1, warps = 4;
    int chunks = 1, chunk_rows = 0;  // of a kv head's query rows
};
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

template <int DP, int NT, bool F8>
nvfp4_status launch_tile(const AttnParams& a, int grid, cudaStream_t stream) {
    using T = TileShape<DP, NT, F8>;
    TileParams p;
    static_cast<AttnParams&>(p) = a;
    p.wide_box = T::kBoxes > 1 && p.D * T::kES % T::kBoxBytes == 0;
    p.tall_box = T::kHalves > 1 && p.page % T::kKeys == 0;
    for (int i = 0; i < 2; ++i) {
        const uint64_t row = static_cast<uint64_t>(p.D) * T::kES, page = row * p.page;
        const uint64_t piece = T::kBoxBytes / T::kES, pieces = p.wide_box ? p.D / piece : 1;
        const uint64_t dims[5] = {p.wide_box ? piece : static_cast<uint64_t>(p.D), static_cast<uint64_t>(p.page), pieces,
                                  static_cast<uint64_t>(p.hk), static_cast<uint64_t>(p.pages)};
        const uint64_t strides[4] = {row, p.wide_box ? T::kBoxBytes : row, page,
                                     p.pages > 1 ? static_cast<uint64_t>(p.page_stride[i]) * T::kES : page * p.hk};
        const uint32_t box[5] = {static_cast<uint32_t>(piece), static_cast<uint32_t>(p.tall_box ? T::kKeys : 16),
                                 static_cast<uint32_t>(p.wide_box ? T::kBoxes : 1), 1, 1};
        if (!host_encode_map(&p.map[i], F8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, p.cache[i], dims,
                             strides, box, T::kBoxBytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return NVFP4_ERR_UNSUPPORTED;
    }
    const size_t smem = 1024 + T::kMain + (T::kQRegs ? 0 : static_cast<size_t>(p.row_blocks) * NT * T::kQ * 256);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(paged_attention_tile_kernel<DP, NT, F8>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return host_cuda_fail(e);
    }
    return launch(paged_attention_tile_kernel<DP, NT, F8>, dim3(grid), dim3(T::kWarps * 32), smem, stream, p);
}

template <bool F8>
nvfp4_status dispatch_tile(const TilePlan& t, const AttnParams& p, int grid, cudaStream_t stream) {
    if (t.dp == 256) return launch_tile<256, 1, F8>(p, grid, stream);
    if (t.dp == 128)
        return t.nt == 1 ? launch_tile<128, 1, F8>(p, grid, stream) : t.nt == 2 ? launch_tile<128, 2, F8>(p, grid, stream)
                                                                                : launch_tile<128, 4, F8>(p, grid, stream);
    return t.nt == 1 ? launch_tile<64, 1, F8>(p, grid, stream) : t.nt == 2 ? launch_tile<64, 2, F8>(p, grid, stream)
                                                                           : launch_tile<64, 4, F8>(p, grid, stream);
}

bool sizes_ok(int seqs, int rows, int hq, int hk, int dim) {
    return seqs >= 0 && rows >= 0 && rows <= kMaxRows && hq >= 0 && hk >= 0 && dim >= 0 && (hk == 0 ? hq == 0 : hq % hk == 0);
}

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
    using namespace nvfp4;
    using namespace nvfp4::ops;
    if (!a) return NVFP4_ERR_NULL;
    if (!sizes_ok(a->seqs, a->rows, a->q_heads, a->kv_heads, a->head_dim) || a->pages < 0 || a->max_pages < 0 ||
        a->page_size < 1 || a->window < 0)
        return NVFP4_ERR_SHAPE;
    if ((a->cache_type != NVFP4_BF16 && a->cache_type != NVFP4_E4M3) ||
        (a->cache_type == NVFP4_BF16 && (a->k_scale || a->v_scale)))
        return NVFP4_ERR_DTYPE;
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
    p.fp8 = a->cache_type == NVFP4_E4M3; p.scale = a->scale;
    const int rows_all = p.rows * p.group, es = p.fp8 ? 1 : 2;
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
        return p.fp8 ? dispatch_tile<true>(t, p, grid, st) : dispatch_tile<false>(t, p, grid, st);
    }
    return launch(paged_attention_scalar_kernel, dim3(a->seqs * a->rows, a->q_heads), dim3(kScalarWarps * 32), 0,
                  static_cast<cudaStream_t>(stream), p);
}
