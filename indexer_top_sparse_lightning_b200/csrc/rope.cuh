// rope.cuh -- per-head RMS norm of queries and keys with the position rotation
// in the same pass; each key goes to its token's row of the paged cache.
//
// For one row x of D elements (a query head, or a token's key) at position p:
//   y_i = x_i * gamma_i / sqrt(mean_{j < n} x_j^2 + eps)   for i < n, else x_i
// then the elements [r0, r0 + R) are rotated in pairs by the angles p * f_i:
//   (a, b) -> (a cos - b sin, b cos + a sin)
// with pairs (i, i + R/2) ("halves") or (2i, 2i + 1) ("interleaved").
//
// What bounds it: memory.  Each row is read once and written once (D * 2 bytes
// each way); the arithmetic is a few operations per element.  8192 tokens of 128 heads of
// 576 with their keys take 462 to 471 us, 5.2 TB/s of the 6.56 of a plain copy (three blocks per SM, at
// 80 registers, spill 40 bytes; four were slower).  A decode step
// is bound by the call: 32 tokens take 7 us on the device, 11.8 with the host's work.  (The launch
// is a programmatic dependent, so that it is ready when the kernel before ends: 1000 ragged tokens
// of 64 heads in a row 15.6 -> 13.4 us.)
//
// Layout.  Eight lanes share a row, 16 bytes (8 elements) per lane and round,
// so a round of the eight lanes is one 128-byte line and a row of D elements
// takes NV = ceil(D / 64) rounds: 576 elements are exactly 9 rounds with every
// lane busy, where a whole warp per row would leave 7/32 of its loads empty.
// All rounds of a row are loaded before anything is computed (9 loads in flight
// per lane), the sum of squares is joined by three shuffles, and the values
// stay in registers until they are stored.  The partner of a halves pair lies
// in another lane's vector; it is loaded again (it is in L1), which keeps the
// kernel free of any rule on where the rotated elements start.
//
// The angle p * f is formed, and brought to [-pi, pi], in 64 bits: at position
// 1e6 a 32-bit product is off by 0.03 radians.  A 64-bit product of an integer
// below 2^31 and a 24-bit fraction is off by 2^-53 of itself, and the sine and
// cosine of the remainder are taken in 32 bits.  The table of a token's angles
// is made once per block and used by all of its rows.
#pragma once
#include <cuda_bf16.h>

#include "common.h"
#include "paging.cuh"
#include "ptx.cuh"

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeGroups = kRopeThreads / 8;   // rows in flight per block
constexpr int kRopeMaxDim = 1024;
constexpr int kRopeTable = 2048;                // (cos, sin) pairs of a block's tokens

struct RopeParams {
    const int32_t* seq_lens;
    const int32_t* cu_q;
    const int32_t* block_table;
    const int32_t* positions;   // [T] rotation positions, or null (the token's place in its sequence)
    const uint16_t* q;          // [T, H, D] bf16 bits, strides in elements
    const uint16_t* k;          // [T, D]
    int64_t q_stride_t, q_stride_h, k_stride_t;
    const float* q_gamma;
    const float* k_gamma;
    const float* inv_freq;      // [R / 2]
    uint16_t* q_out;            // [T, H, D] dense
    void* k_cache;              // bf16 rows, or e4m3 codes with k_scale
    float* k_scale;             // [rows, 5]
    uint32_t* status;
    int32_t B, T, H, D, max_blocks, num_blocks;
    int32_t q_norm, k_norm, r0, R, interleaved, fp8;
    float eps;
    int32_t q_blocks;           // blocks of query rows; the key blocks follow
    int32_t tpc, hpc, hsplit;   // query blocks: tokens per block, heads per block, blocks per token group
    int32_t ktpc;               // key blocks: tokens per block
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Lane `gl` (0..7) of a row's eight lanes.  `x` is the row; loads first, so that
// the caller can place them before the block's angles are ready.
template <int NV>
__device__ __forceinline__ void rope_load(const uint16_t* x, int D, int gl, uint4 (&raw)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * 8 + gl) * 8;
        raw[i] = e < D ? *reinterpret_cast<const uint4*>(x + e) : make_uint4(0u, 0u, 0u, 0u);
    }
}

// 1 / sqrt(mean square + eps) of a row's leading `norm` elements (1 without a
// norm); `lanes` is the mask of the row's eight lanes.
template <int NV>
__device__ __forceinline__ float row_rstd(const uint4 (&raw)[NV], int norm, float eps, int gl, uint32_t lanes) {
    if (norm <= 0) return 1.0f;
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float f[8];
        unpack8(raw[i], f);
        if ((i * 8 + gl) * 8 < norm)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) ss += __shfl_xor_sync(lanes, ss, d);
    return 1.0f / sqrtf(ss / (float)norm + eps);
}

// The elements e..e+7 of a row, normalized (without the rotation).
__device__ __forceinline__ void scaled8(uint4 v, int e, const float* gamma, int norm, float rstd, float (&f)[8]) {
    unpack8(v, f);
    if (e < norm) {
        const float4 g0 = __ldg(reinterpret_cast<const float4*>(gamma + e));
        const float4 g1 = __ldg(reinterpret_cast<const float4*>(gamma + e) + 1);
        const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] * rstd * g[j];
    }
}

// The results e..e+7 of row x: normalized and, inside [r0, r0 + R), rotated.
__device__ __forceinline__ void turned8(const uint16_t* x, uint4 v, int e, const float* gamma, int norm, float rstd,
                                        const RopeParams& p, const float2* cs, float (&f)[8]) {
    scaled8(v, e, gamma, norm, rstd, f);
    const int o = e - p.r0;
    if (o < 0 || o >= p.R) return;
    if (p.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 c = cs[o / 2 + j];
            const float a = f[2 * j], b = f[2 * j + 1];
            f[2 * j] = a * c.x - b * c.y;
            f[2 * j + 1] = b * c.x + a * c.y;
        }
    } else {
        const int half = p.R / 2;
        const bool low = o < half;
        const int pe = low ? e + half : e - half;
        const int t0 = low ? o : o - half;
        float g[8];
        scaled8(*reinterpret_cast<const uint4*>(x + pe), pe, gamma, norm, rstd, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 c = cs[t0 + j];
            f[j] = f[j] * c.x + (low ? -g[j] : g[j]) * c.y;
        }
    }
}

// Blocks [0, q_blocks): query rows (tpc tokens x hpc heads each, eight lanes a
// row, kRopeGroups rows at a time); the blocks behind them: the key rows of
// ktpc tokens each.  Query blocks of one token's heads share its angle table.
template <int NV>
__global__ void __launch_bounds__(kRopeThreads, NV <= 2 ? 6 : NV <= 4 ? 4 : NV <= 9 ? 3 : 2)
    qk_norm_rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 s_cs[kRopeTable];
    __shared__ int s_seq[kRopeGroups];
    __shared__ int64_t s_pos[kRopeGroups];   // the token's place in its sequence
    const int gl = threadIdx.x & 7, group = threadIdx.x >> 3;
    const uint32_t lanes = 0xFFu << (threadIdx.x & 24);
    const bool keys = (int)blockIdx.x >= p.q_blocks;
    const int unit = keys ? (int)blockIdx.x - p.q_blocks : (int)blockIdx.x;
    const int t0 = keys ? unit * p.ktpc : unit / p.hsplit * p.tpc;
    const int h0 = keys ? 0 : unit % p.hsplit * p.hpc;
    const int hn = keys ? 1 : (p.H - h0 < p.hpc ? p.H - h0 : p.hpc);
    const int per = keys ? p.ktpc : p.tpc;
    const int tn = p.T - t0 < per ? p.T - t0 : per;
    const int rows = tn * hn;
    auto row_ptr = [&](int r) -> const uint16_t* {
        const int64_t t = t0 + r / hn;
        return keys ? p.k + t * p.k_stride_t : p.q + t * p.q_stride_t + (int64_t)(h0 + r % hn) * p.q_stride_h;
    };
    griddep_wait();
    // the first rows' loads go out before the angles are made
    uint4 raw[NV];
    if (group < rows) rope_load<NV>(row_ptr(group), p.D, gl, raw);

    if ((int)threadIdx.x < tn) {
        const int t = t0 + (int)threadIdx.x;
        const int b = query_sequence(p.cu_q, p.B, t);
        s_seq[threadIdx.x] = b;
        s_pos[threadIdx.x] = b < 0 ? 0 : (int64_t)__ldg(p.seq_lens + b) - __ldg(p.cu_q + b + 1) + t;
    }
    __syncthreads();
    const int half = p.R / 2;
    for (int i = threadIdx.x; i < tn * half; i += kRopeThreads) {
        const int lt = i / half, j = i - lt * half;
        const double pos = p.positions ? (double)__ldg(p.positions + t0 + lt) : (double)s_pos[lt];
        const double a = pos * (double)__ldg(p.inv_freq + j);
        const double turns = rint(a * 0.15915494309189533577);
        float s, c;
        sincosf((float)fma(-turns, 6.283185307179586477, a), &s, &c);
        s_cs[i] = make_float2(c, s);
    }
    __syncthreads();

    for (int r = group; r < rows; r += kRopeGroups) {
        const uint16_t* x = row_ptr(r);
        if (r != group) rope_load<NV>(x, p.D, gl, raw);
        const int lt = r / hn;
        if (s_seq[lt] < 0) continue;              // a row behind the last sequence stays as it was
        const float2* cs = s_cs + lt * half;
        const float* gamma = keys ? p.k_gamma : p.q_gamma;
        const int norm = keys ? p.k_norm : p.q_norm;
        const float rstd = row_rstd<NV>(raw, norm, p.eps, gl, lanes);
        int64_t row = 0;
        if (keys) {
            row = cache_row(p.block_table, p.max_blocks, p.num_blocks, s_seq[lt], s_pos[lt]);
            if (row < 0) {
                if (gl == 0) atomicCAS(p.status, 0u, (uint32_t)kStBounds);
                continue;
            }
        }
        if (!keys || !p.fp8) {
            uint16_t* y = keys ? static_cast<uint16_t*>(p.k_cache) + row * p.D
                               : p.q_out + ((int64_t)(t0 + lt) * p.H + h0 + r % hn) * p.D;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * 8 + gl) * 8;
                if (e < p.D) {
                    float f[8];
                    turned8(x, raw[i], e, gamma, norm, rstd, p, cs, f);
                    raw[i] = pack8(f);
                }
            }
            // q_out may be q itself: every lane of the row has read its values
            __syncwarp(lanes);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * 8 + gl) * 8;
                if (e < p.D) *reinterpret_cast<uint4*>(y + e) = raw[i];
            }
        } else if constexpr (NV == 9) {
            // e4m3 rows with one scale per 128 elements: two rounds of the eight lanes are a
            // tile, the last tile being the 64 behind the latent.  The scale is taken from,
            // and the codes rounded from, the 32-bit values: one rounding per element.
            uint8_t* y = static_cast<uint8_t*>(p.k_cache) + row * kDqk;
#pragma unroll
            for (int t = 0; t < 5; ++t) {
                float v[2][8], am = 0.0f;
#pragma unroll
                for (int u = 0; u < 2 && 2 * t + u < NV; ++u) {
                    turned8(x, raw[2 * t + u], ((2 * t + u) * 8 + gl) * 8, gamma, norm, rstd, p, cs, v[u]);
#pragma unroll
                    for (int j = 0; j < 8; ++j) am = fmaxf(am, fabsf(v[u][j]));
                }
#pragma unroll
                for (int d = 4; d > 0; d >>= 1) am = fmaxf(am, __shfl_xor_sync(lanes, am, d));
                float sc = am / 448.0f;
                if (!(sc > 0.0f)) sc = 1.0f;      // a tile of zeros (or of values too small for a scale)
                if (gl == 0) p.k_scale[row * 5 + t] = sc;
#pragma unroll
                for (int u = 0; u < 2 && 2 * t + u < NV; ++u) {
                    uint32_t w[2] = {0u, 0u};
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        uint16_t c;
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(v[u][j + 1] / sc), "f"(v[u][j] / sc));
                        // a zero is stored as +0
                        if (!(c & 0x007Fu)) c &= 0xFF00u;
                        if (!(c & 0x7F00u)) c &= 0x00FFu;
                        w[j / 4] |= (uint32_t)c << (8 * (j & 2));
                    }
                    *reinterpret_cast<uint2*>(y + ((2 * t + u) * 8 + gl) * 8) = make_uint2(w[0], w[1]);
                }
            }
        }
    }
}

}  // namespace dsa
