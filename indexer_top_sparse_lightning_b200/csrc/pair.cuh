// pair.cuh -- helpers of the attention kernels, which run as clusters of two
// CTAs ("pairs") over contiguous shares of a list of blocks.
#pragma once
#include "common.h"
#include "ptx.cuh"

namespace dsa {

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 operations in one instruction, each rounded by itself.
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
        "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// Arrive on an mbarrier of CTA 0 of the pair (a local arrive when this is CTA 0).
__device__ __forceinline__ void arrive_leader(uint64_t* bar, uint32_t crank) {
    if (crank == 0) mbar_arrive(bar);
    else mbar_arrive_remote(mapa_shared(smem_u32(bar), 0));
}

// The contiguous block range of pair `pr` among `np` pairs: [g0, g1) of `total`.
__device__ __forceinline__ int64_t pair_start(int64_t total, int pr, int np) { return total * pr / np; }
// The pair whose range holds global block g.
__device__ __forceinline__ int pair_of_block(int64_t total, int64_t g, int np) {
    return (int)(((g + 1) * np + total - 1) / total) - 1;
}

}  // namespace dsa
