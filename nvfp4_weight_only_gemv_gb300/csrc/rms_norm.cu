// Root-mean-square norm of rows, with the residual's addition in front and an 8-bit form behind.
//
//   h = x + residual          (fp32; residual_out = h in the residual's type)
//   y = h / sqrt(mean(h^2) + eps) * weight
//   E4M3 output: s = max(max|y| / 448, 2^-64) per row or per group of columns (to a unit in the last place),
//                code = E4M3(y / s), an fp32 quotient by this s
//
// The row stays in registers between the sum of squares and the store, so every operand is read
// once and every result written once: the kernel is bound by that traffic for many rows and by one
// chain of load, reduction and store for few.

#include "ops_common.cuh"

#include <type_traits>

namespace nvfp4 {
namespace {

using namespace ops;

constexpr int kMaxCols = 32768;  // 1024 threads x 4 chunks of 8 columns
constexpr float kScaleFloor = 5.421010862427522e-20f;  // 2^-64: its reciprocal is finite

struct NormParams {
    const void* x;
    const void* residual;
    const void* weight;
    void* residual_out;
    void* y;
    float* scales;
    int64_t ldx, ldr, ldro, ldy;
    int w_type, y_type;
    int rows, cols, group;  // group: columns per scale
    int tpr_log2;           // threads per row (vector kernel)
    float eps;
    float shrink, mean_of;  // see add_square
};

// The larger magnitude, NaN if either is: a NaN reaches the scale, as the quotient's definition wants.
__device__ __forceinline__ float max_mag(float m, float v) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(m), "f"(fabsf(v)));
    return d;
}

__device__ __forceinline__ float scale_of(float amax) {
    const float s = amax * (1.0f / 448.0f);
    return s < kScaleFloor ? kScaleFloor : s;  // NaN stays NaN
}
// Quotients by a scale, at most 448 in magnitude. (8192 rows, one scale a row: 4096 columns 42.2 us, 16384 columns
// 260; with a division per value 51.1 and 296; with the product alone 43.6 and 250.)
struct Scaled {
    float inv, s;
    __device__ __forceinline__ Scaled() {}
    __device__ __forceinline__ explicit Scaled(float scale) {
        asm("rcp.approx.f32 %0, %1;" : "=f"(inv) : "f"(scale));  // to a unit in the last place: a scale is 2^-64 or more
        s = scale < INFINITY ? scale : 0.0f;                    // infinity: a finite y over it is zero; NaN stays in inv
    }
    __device__ __forceinline__ float operator()(float y) const { return put_right(y * inv, y, s, inv); }
};

template <typename RT>
struct HasResidual { static constexpr bool value = true; };
template <>
struct HasResidual<void> { static constexpr bool value = false; };

// mean(h^2) = sum((h * shrink)^2) * mean_of, shrink = the power of two at or below 1 / sqrt(cols):
// the sum stays in range wherever a single square does, at one exact product per value.
__device__ __forceinline__ float add_square(float h, float shrink, float sum) {
    const float t = h * shrink;
    return fmaf(t, t, sum);
}

// Sum (or integer maximum) over the threads of one row: shuffles, then shared memory where a row
// has more than one warp. Fixed order.
__device__ __forceinline__ float row_sum(float v, int tpr, float* red, int row_in_cta) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = tpr >> 5, first = row_in_cta * warps;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < warps; ++i) s += red[first + i];
    return s;
}

__device__ __forceinline__ float row_max(float v, int tpr, float* red, int row_in_cta) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = max_mag(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = tpr >> 5, first = row_in_cta * warps;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    float m = 0.0f;
    for (int i = 0; i < warps; ++i) m = max_mag(m, red[first + i]);
    return m;
}

// Vector form: tpr threads a row, each with CH chunks of 8 columns.
template <typename XT, typename RT, int CH, bool Q8>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float red[32];
    __shared__ float redm[32];
    pdl_launch_dependents();
    const int tpr = 1 << p.tpr_log2;
    const int row_in_cta = threadIdx.x >> p.tpr_log2, t = threadIdx.x & (tpr - 1);
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> p.tpr_log2) + row_in_cta;
    const int chunks = p.cols >> 3;
    const bool live = row < p.rows;
    pdl_wait();
    float h[CH][8];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = t + j * tpr;
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = 0.0f;
        if (live && c < chunks) {
            load_vec(static_cast<const XT*>(p.x) + row * p.ldx + c * 8, h[j]);
            if constexpr (HasResidual<RT>::value) {
                float r[8];
                load_vec(static_cast<const RT*>(p.residual) + row * p.ldr + c * 8, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] += r[i];
            }
        }
    }
    auto load_weight = [&](int c, float (&v)[8]) {
        if (p.w_type == NVFP4_F32) load_vec(static_cast<const float*>(p.weight) + c * 8, v);
        else load_vec(static_cast<const __nv_bfloat16*>(p.weight) + c * 8, v);
    };
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if constexpr (HasResidual<RT>::value) {
            const int c = t + j * tpr;
            if (live && c < chunks) store_vec(static_cast<RT*>(p.residual_out) + row * p.ldro + c * 8, h[j]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = add_square(h[j][i], p.shrink, sum);
    }
    const float rstd = rsqrtf(fmaf(row_sum(sum, tpr, red, row_in_cta), p.mean_of, p.eps));
    float amax[CH];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        amax[j] = 0.0f;
        if (t + j * tpr >= chunks) continue;  // h is zero there
        // behind the sum: requested before it, the weights' registers cost more occupancy than their
        // latency (8192 x 4096: 48 us)
        float w[8];
        load_weight(t + j * tpr, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            h[j][i] = h[j][i] * rstd * w[i];
            if constexpr (Q8) amax[j] = max_mag(amax[j], h[j][i]);
        }
    }
    if constexpr (!Q8) {
        if (p.y_type == NVFP4_F32) {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (live && t + j * tpr < chunks) store_vec(static_cast<float*>(p.y) + row * p.ldy + (t + j * tpr) * 8, h[j]);
        } else {
#pragma unroll
            for (int j = 0; j < CH; ++j)
                if (live && t + j * tpr < chunks) store_vec(static_cast<__nv_bfloat16*>(p.y) + row * p.ldy + (t + j * tpr) * 8, h[j]);
        }
        return;
    }
    Scaled over[CH];
    if (p.group == p.cols) {
        float top = amax[0];
#pragma unroll
        for (int j = 1; j < CH; ++j) top = max_mag(top, amax[j]);
        const float s = scale_of(row_max(top, tpr, redm, row_in_cta));
        if (live && t == 0) p.scales[row] = s;
#pragma unroll
        for (int j = 0; j < CH; ++j) over[j] = Scaled(s);
    } else {
        // a group of 16..256 columns is 2..32 neighbouring lanes
        for (int o = 1; o < p.group >> 3; o <<= 1) {
#pragma unroll
            for (int j = 0; j < CH; ++j) amax[j] = max_mag(amax[j], __shfl_xor_sync(0xffffffffu, amax[j], o));
        }
        const int lanes_log2 = __ffs(p.group >> 3) - 1;
        float* const out = p.scales + row * (chunks >> lanes_log2);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int c = t + j * tpr;
            const float s = scale_of(amax[j]);
            over[j] = Scaled(s);
            if (live && c < chunks && (c & ((p.group >> 3) - 1)) == 0) out[c >> lanes_log2] = s;
        }
    }
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = t + j * tpr;
        if (!live || c >= chunks) continue;
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = pack_e4m3(over[j](h[j][2 * i]), over[j](h[j][2 * i + 1]));
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.y) + row * p.ldy + c * 8) = make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
    }
}

__device__ __forceinline__ float load_typed(const void* p, int type, int64_t i) {
    return type == NVFP4_F32 ? static_cast<const float*>(p)[i] : load_one(static_cast<const __nv_bfloat16*>(p) + i);
}

// Any alignment and any number of columns: one CTA a row, h in shared memory, one value at a time.
template <typename XT, typename RT>
__global__ void __launch_bounds__(256) rms_norm_scalar_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ float h[];
    __shared__ float red[32];
    __shared__ float redm[32];
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x;
    const int t = threadIdx.x, n = blockDim.x;
    float sum = 0.0f;
    for (int c = t; c < p.cols; c += n) {
        float v = load_one(static_cast<const XT*>(p.x) + row * p.ldx + c);
        if constexpr (HasResidual<RT>::value) {
            v += load_one(static_cast<const RT*>(p.residual) + row * p.ldr + c);
            if constexpr (sizeof(RT) == 4) static_cast<float*>(p.residual_out)[row * p.ldro + c] = v;
            else static_cast<__nv_bfloat16*>(p.residual_out)[row * p.ldro + c] = __float2bfloat16_rn(v);
        }
        h[c] = v;
        sum = add_square(v, p.shrink, sum);
    }
    const float rstd = rsqrtf(fmaf(row_sum(sum, n, red, 0), p.mean_of, p.eps));
    float amax = 0.0f;
    for (int c = t; c < p.cols; c += n) {
        const float v = h[c] * rstd * load_typed(p.weight, p.w_type, c);
        h[c] = v;
        amax = max_mag(amax, v);
        if (p.y_type == NVFP4_F32) static_cast<float*>(p.y)[row * p.ldy + c] = v;
        else if (p.y_type == NVFP4_BF16) static_cast<__nv_bfloat16*>(p.y)[row * p.ldy + c] = __float2bfloat16_rn(v);
    }
    if (p.y_type != NVFP4_E4M3) return;
    uint8_t* const y = static_cast<uint8_t*>(p.y) + row * p.ldy;
    if (p.group == p.cols) {
        const float s = scale_of(row_max(amax, n, redm, 0));
        const Scaled over(s);
        if (t == 0) p.scales[row] = s;
        for (int c = t; c < p.cols; c += n) y[c] = static_cast<uint8_t>(pack_e4m3(over(h[c]), 0.0f));
        return;
    }
    __syncthreads();  // h is complete; a warp takes a group
    for (int g = t >> 5; g < p.cols / p.group; g += n >> 5) {
        float m = 0.0f;
        for (int c = g * p.group + (t & 31); c < (g + 1) * p.group; c += 32) m = max_mag(m, h[c]);
        const float s = scale_of(row_max(m, 32, redm, 0));
        const Scaled over(s);
        if ((t & 31) == 0) p.scales[row * (p.cols / p.group) + g] = s;
        for (int c = g * p.group + (t & 31); c < (g + 1) * p.group; c += 32) y[c] = static_cast<uint8_t>(pack_e4m3(over(h[c]), 0.0f));
    }
}

template <typename XT, typename RT>
nvfp4_status run(const NormParams& in, bool vec, cudaStream_t stream) {
    NormParams p = in;
    if (!vec) {
        const size_t smem = static_cast<size_t>(p.cols) * 4;
        if (smem > 40 * 1024) {
            const cudaError_t e = cudaFuncSetAttribute(rms_norm_scalar_kernel<XT, RT>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxCols * 4);
            if (e != cudaSuccess) return host_cuda_fail(e);
        }
        return launch(rms_norm_scalar_kernel<XT, RT>, dim3(p.rows), dim3(256), smem, stream, p);
    }
    // Few rows: a chunk a thread, the shortest chain. Many: 2 chunks a thread, so that the sum over the
    // row's threads and its barrier are paid for once per 16 values (8192 x 4096 bf16: 43.2 us with 1, 40.2 with
    // 2, 45.4 with 4).
    const int chunks = p.cols / 8, most = p.rows >= 2 * host_sm_count() ? 2 : 1;
    int lg = 5;
    while (lg < 10 && (most << lg) < chunks) ++lg;
    p.tpr_log2 = lg;
    const int tpr = 1 << lg, threads = tpr < 128 ? 128 : tpr, rpc = threads / tpr;
    const dim3 grid((p.rows + rpc - 1) / rpc), block(threads);
    const int ch = (chunks + tpr - 1) / tpr;
    auto go = [&](auto q8) {
        constexpr bool Q8 = decltype(q8)::value;
        if (ch <= 1) return launch(rms_norm_kernel<XT, RT, 1, Q8>, grid, block, 0, stream, p);
        if (ch <= 2) return launch(rms_norm_kernel<XT, RT, 2, Q8>, grid, block, 0, stream, p);
        return launch(rms_norm_kernel<XT, RT, 4, Q8>, grid, block, 0, stream, p);
    };
    return p.y_type == NVFP4_E4M3 ? go(std::true_type{}) : go(std::false_type{});
}

template <typename XT>
nvfp4_status run_x(const NormParams& p, int r_type, bool vec, cudaStream_t stream) {
    if (!p.residual) return run<XT, void>(p, vec, stream);
    return r_type == NVFP4_F32 ? run<XT, float>(p, vec, stream) : run<XT, __nv_bfloat16>(p, vec, stream);
}

bool wide_type(int t) { return t == NVFP4_F32 || t == NVFP4_BF16; }

}  // namespace
}  // namespace nvfp4

extern "C" nvfp4_status nvfp4_rms_norm(const nvfp4_rms_norm_args* a, void* stream) {
    using namespace nvfp4;
    using namespace nvfp4::ops;
    if (!a) return NVFP4_ERR_NULL;
    if (a->rows < 0 || a->cols < 0 || !(a->eps >= 0.0f)) return NVFP4_ERR_SHAPE;
    if (!wide_type(a->x_type) || !wide_type(a->w_type) || (a->residual && !wide_type(a->residual_type)) ||
        !(wide_type(a->y_type) || a->y_type == NVFP4_E4M3))
        return NVFP4_ERR_DTYPE;
    const bool e4m3 = a->y_type == NVFP4_E4M3;
    if (e4m3 && a->group != 0 &&
        (a->group < 16 || a->group > 256 || (a->group & (a->group - 1)) || a->cols % a->group))
        return NVFP4_ERR_SHAPE;
    if (!e4m3 && a->group != 0) return NVFP4_ERR_SHAPE;
    if (a->rows == 0 || a->cols == 0) return NVFP4_OK;
    if (a->cols > kMaxCols) return NVFP4_ERR_UNSUPPORTED;
    if (!a->x || !a->weight || !a->y || (a->residual && !a->residual_out) || (e4m3 && !a->scales)) return NVFP4_ERR_NULL;
    // rows that are read may overlap or repeat; rows that are written may not
    if (a->ldx < 0 || (a->residual && a->ldr < 0) || (a->rows > 1 && (a->ldy < a->cols || (a->residual && a->ldro < a->cols))))
        return NVFP4_ERR_SHAPE;
    NormParams p{};
    p.x = a->x; p.residual = a->residual; p.weight = a->weight; p.residual_out = a->residual_out; p.y = a->y;
    p.scales = a->scales;
    p.ldx = a->ldx; p.ldr = a->ldr; p.ldro = a->ldro; p.ldy = a->ldy;
    p.w_type = a->w_type; p.y_type = a->y_type;
    p.rows = a->rows; p.cols = a->cols; p.group = e4m3 && a->group ? a->group : a->cols;
    p.eps = a->eps;
    int half_log2 = 0;
    while ((1 << 2 * half_log2) < p.cols) ++half_log2;
    p.shrink = 1.0f / static_cast<float>(1 << half_log2);
    p.mean_of = static_cast<float>(static_cast<double>(1ll << 2 * half_log2) / p.cols);
    // Vectors of 8: rows, and the row pitch, on 16-byte boundaries (8 for the codes).
    auto fits = [](const void* q, int64_t ld, int type) {
        const int bytes = type == NVFP4_E4M3 ? 8 : 16;
        return aligned(q, bytes) && (ld * type_bytes(type)) % bytes == 0;
    };
    const bool vec = p.cols % 8 == 0 && fits(p.x, p.ldx, a->x_type) && fits(p.y, p.ldy, a->y_type) &&
                     aligned(p.weight, 16) &&
                     (!p.residual || (fits(p.residual, p.ldr, a->residual_type) &&
                                      fits(p.residual_out, p.ldro, a->residual_type)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a->x_type == NVFP4_F32 ? run_x<float>(p, a->residual_type, vec, st)
                                  : run_x<__nv_bfloat16>(p, a->residual_type, vec, st);
}
