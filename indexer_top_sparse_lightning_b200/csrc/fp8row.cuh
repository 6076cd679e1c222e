// fp8row.cuh -- decoding of FP8 latent rows (e4m3 codes, one fp32 scale per
// 128-element tile) to bf16, shared by the staging kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace dsa {

constexpr int kKvTiles = 5;   // 4 latent tiles of 128 + the 64-element RoPE tile

// Two e4m3 codes (low byte first) -> two floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t two) {
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(two));
    return __half22float2(*reinterpret_cast<__half2*>(&h2));
}

// Dequantizes one 16-code chunk (tile scale s) into 16 bf16 values at dst.
__device__ __forceinline__ void stage_chunk(uint4 raw, float s, uint4* dst) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 lo = e4m3x2_to_float2((uint16_t)(w[k] & 0xFFFFu));
        const float2 hi = e4m3x2_to_float2((uint16_t)(w[k] >> 16));
        const __nv_bfloat162 a = __floats2bfloat162_rn(lo.x * s, lo.y * s);
        const __nv_bfloat162 b = __floats2bfloat162_rn(hi.x * s, hi.y * s);
        o[2 * k] = *reinterpret_cast<const uint32_t*>(&a);
        o[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&b);
    }
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace dsa
