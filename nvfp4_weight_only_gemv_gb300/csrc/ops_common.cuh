// What the decode step's operators around the products share: conversions, launch attributes and
// the host state that lives beside the GEMV entry points (nvfp4_gemv.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4_gemv.h"

namespace nvfp4 {

// Host state kept by nvfp4_gemv.cu.
bool host_pdl_enabled();                       // nvfp4_set_pdl
int host_variant();                            // nvfp4_set_variant
nvfp4_status host_cuda_fail(cudaError_t e);    // records e for nvfp4_last_cuda_error
int host_sm_count();                           // SMs of the current device, 0 on an error
uint64_t host_wait_ns();                       // nvfp4_set_wait_budget_ns
// Encodes a tiled tensor map (unit element strides, no interleave, zero fill).
bool host_encode_map(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* base, const uint64_t* dims,
                     const uint64_t* strides, const uint32_t* box, CUtensorMapSwizzle swizzle);

// Where the current device's status word stands, which nvfp4_device_status reads; NULL on an error, which is recorded.
// Device symbols are not shared between translation units, so the operators' kernels get it with their arguments: with a
// word of each unit's own nvfp4_device_status waited for a copy of each, 77 us for six.
int* host_status_word();
// Reads and clears the word that paged_attention.cu has of its own (see status_word there), which gives its function when the
// library is loaded; NULL where nvfp4_gemv.cu is built alone.
using StatusReader = cudaError_t (*)(int* bits);
bool set_attention_status(StatusReader reader);

namespace ops {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float bf16_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// Two floats to bf16x2, round to nearest even, `lo` in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two floats to E4M3 codes (low byte = lo), to nearest even, beyond 448 to 448; NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two E4M3 codes to f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t codes) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(codes)));
    return d;
}

// The 4-bit cache: 16 keys (or values) of a kv head are a record of 9 D bytes: E2M1 codes [16][D / 2], element
// 2j in the low nibble of byte j, then the E4M3 scales of 16 elements each, [D / 16][16 keys]. So a key's
// codes are whole bytes of its own, which tokens appended side by side can store, any number of records in a
// page is one contiguous copy, and a lane of the attention kernel finds the scales of its four values' keys in
// one word.
constexpr int kRecordKeys = 16;
__host__ __device__ constexpr int64_t record_bytes(int dim) { return 9ll * dim; }

// Eight E2M1 codes (element 2i in the low nibble of byte i) to four f16x2, low half = even element (exact).
__device__ __forceinline__ void e2m1x8_f16x2(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        " cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// Eight floats to E2M1 codes (element 0 in the lowest nibble), to nearest, ties to the even code, beyond 6 to 6.
__device__ __forceinline__ uint32_t pack_e2m1x8(const float* v) {
    uint32_t d;
    asm("{\n .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n}"
        : "=r"(d)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return d;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_f16x2(code & 0xffu) & 0xffffu)));
}

// A quotient x / s from q = x * inv, inv near 1 / s: q put right by its remainder (P. Markstein, IBM J. Res. Dev.
// 34, 1990). What is stored as E4M3 gets the codes of an fp32 quotient this way (tested against it), at two
// products a value: q alone took the other code for values beside the middle of two.
__device__ __forceinline__ float put_right(float q, float x, float s, float inv) { return fmaf(fmaf(-q, s, x), inv, q); }

template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4 q = *reinterpret_cast<const float4*>(p + i);
        v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
}
__device__ __forceinline__ void unpack_bf16(uint32_t u, float& a, float& b) { a = bf16_lo(u); b = bf16_hi(u); }

// Eight consecutive values of an aligned row, widened.
__device__ __forceinline__ void load_vec(const float* p, float (&v)[8]) { load_f32(p, v); }
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    unpack_bf16(q.x, v[0], v[1]); unpack_bf16(q.y, v[2], v[3]);
    unpack_bf16(q.z, v[4], v[5]); unpack_bf16(q.w, v[6], v[7]);
}
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }

template <int N>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                              pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int type_bytes(int t) { return t == NVFP4_F32 ? 4 : t == NVFP4_BF16 ? 2 : 1; }

// Launches with the programmatic-dependent-launch attribute when nvfp4_set_pdl is on. Every
// thread of these kernels passes griddepcontrol.wait before it touches an operand, so a kernel
// that depends on this one also comes after everything this one came after.
template <typename P>
nvfp4_status launch(void (*kernel)(P), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const P& p) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    if (host_pdl_enabled()) {
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
    }
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? NVFP4_OK : host_cuda_fail(e);
}

}  // namespace ops
}  // namespace nvfp4
