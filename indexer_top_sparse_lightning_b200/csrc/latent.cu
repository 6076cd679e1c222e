// latent.cu -- copies that the dense kernels read in place of an FP8 latent cache:
// the sequences' rows, and queries, as fp16; and the tensor maps over rows.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/dsa.h"
#include "common.h"
#include "fp8row.cuh"
#include "host.h"
#include "ptx.cuh"

namespace dsa {

// The pages of every sequence as fp16: x = code x tile scale / page factor, rounded
// (2^-11 of the value), and the rest x - that, rounded (2^-22 of the value, or 2^-29 of the page's largest
// scale where that is more: fp16's smallest step), in a copy that is laid out by sequence: page i of
// sequence b at b * pages + i.  The page factor is the power of two that brings the
// largest value that the page's scales allow below 2^14; positions behind the
// sequence's end do not count, whatever they hold.  One block per page: its 64 rows
// are 2304 runs of 16 codes, nine per thread, all loaded before any is converted.
// Memory-bound: reads 596 bytes a row and writes 2304.  (Dense attention of few new tokens
// converts in its own kernel instead, chunk_fp8.cuh.)
struct PagesParams {
    const int32_t* seq_lens;
    const int32_t* block_table;
    const uint8_t* codes;       // [num_blocks * 64, 576]
    const float* scale;         // [num_blocks * 64, 5]
    uint16_t* rows;             // [B * pages * 64, 2 x 576] fp16 bits
    float* page_scale;          // [B * pages]
    int32_t B, max_blocks, num_blocks, pages;
};

constexpr int kPagesThreads = 256;

__global__ void __launch_bounds__(kPagesThreads) kv_fp8_pages_kernel(const __grid_constant__ PagesParams p) {
    griddep_launch_dependents();
    __shared__ float s_top[kPagesThreads / 32];
    const int b = (int)blockIdx.x / p.pages, page = (int)blockIdx.x % p.pages;
    const int64_t left = (int64_t)__ldg(p.seq_lens + b) - (int64_t)page * kPage;
    if (left <= 0 || page >= p.max_blocks) return;
    const int id = __ldg(p.block_table + (int64_t)b * p.max_blocks + page);
    if (id < 0 || id >= p.num_blocks) {                // the attention kernel reports it and does not read the copy
        if (threadIdx.x == 0) p.page_scale[blockIdx.x] = 1.0f;
        return;
    }
    constexpr int RUNS = kPage * kDqk / 16, PER = RUNS / kPagesThreads;
    static_assert(RUNS % kPagesThreads == 0, "whole runs per thread");
    const uint4* src = reinterpret_cast<const uint4*>(p.codes + (int64_t)id * kPage * kDqk);
    const float* sc = p.scale + (int64_t)id * kPage * kKvTiles;
    uint4* dst = reinterpret_cast<uint4*>(p.rows + (int64_t)blockIdx.x * kPage * kCopyRow);
    uint4 v[PER];
    float s[PER], top = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = i * kPagesThreads + (int)threadIdx.x;
        v[i] = __ldg(src + r);
        s[i] = __ldg(sc + r / 36 * kKvTiles + r % 36 / 8);
        if (r / 36 < left) top = fmaxf(top, fabsf(s[i]));
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPagesThreads / 32; ++w) top = fmaxf(top, s_top[w]);
    // scales below 2^(E + 1), codes up to 448 < 2^9: value / 2^(E - 4) < 2^14
    int E = (int)(__float_as_uint(top) >> 23) - 127;
    E = top == 0.0f ? 4 : E < -100 ? -100 : E > 120 ? 120 : E;
    const float down = __uint_as_float((uint32_t)(4 - E + 127) << 23);
    if (threadIdx.x == 0) p.page_scale[blockIdx.x] = __uint_as_float((uint32_t)(E - 4 + 127) << 23);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = i * kPagesThreads + (int)threadIdx.x;
        const float f = s[i] * down;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[8], rest[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float2 x = e4m3x2_to_float2((uint16_t)(w[k / 2] >> (16 * (k & 1))));
            const float x0 = x.x * f, x1 = x.y * f;
            const __half2 h = __floats2half2_rn(x0, x1);
            const __half2 l = __floats2half2_rn(x0 - __low2float(h), x1 - __high2float(h));
            o[k] = *reinterpret_cast<const uint32_t*>(&h);
            rest[k] = *reinterpret_cast<const uint32_t*>(&l);
        }
        uint4* d = dst + r / 36 * (kCopyRow / 8) + 2 * (r % 36);
        d[0] = make_uint4(o[0], o[1], o[2], o[3]);
        d[1] = make_uint4(o[4], o[5], o[6], o[7]);
        d[kDqk / 8] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
        d[kDqk / 8 + 1] = make_uint4(rest[4], rest[5], rest[6], rest[7]);
    }
}

// The queries as fp16 rows of q * 2^(13 - E), E the exponent of the row's largest
// magnitude, and the factors 2^(E - 13): exact but for what lies 2^-28 below that
// magnitude.  Eight lanes a row, nine 16-byte pieces each.
constexpr int kQueryThreads = 256;

__global__ void __launch_bounds__(kQueryThreads) q_fp16_kernel(const uint16_t* q, int64_t nrows, uint16_t* out, float* factor) {
    griddep_launch_dependents();
    const int64_t row = (int64_t)blockIdx.x * (kQueryThreads / 8) + (threadIdx.x >> 3);
    const int gl = threadIdx.x & 7;
    const uint32_t lanes = 0xFFu << (threadIdx.x & 24);
    if (row >= nrows) return;
    constexpr int PER = kDqk / 64;
    const uint4* src = reinterpret_cast<const uint4*>(q + row * kDqk);
    uint4 v[PER];
    uint32_t top = 0;                                   // bf16 magnitudes compare as integers
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        v[i] = src[8 * i + gl];
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
    }
#pragma unroll
    for (int d = 4; d > 0; d >>= 1) top = max(top, __shfl_xor_sync(lanes, top, d));
    int E = (int)(top >> 7) - 127;
    E = E < -100 ? -100 : E > 127 ? 127 : E;
    const float down = __uint_as_float((uint32_t)(13 - E + 127) << 23);
    uint4* dst = reinterpret_cast<uint4*>(out + row * kDqk);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w[e] << 16) * down, __uint_as_float(w[e] & 0xFFFF0000u) * down);
            o[e] = *reinterpret_cast<const uint32_t*>(&h);
        }
        dst[8 * i + gl] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (gl == 0) factor[row] = __uint_as_float((uint32_t)(E - 13 + 127) << 23);
}

namespace host {

dsa_status copy_fp8_pages(const dsa_batch* bt, const dsa_attn_inputs* at, int64_t pages, void* rows, float* page_scale,
                          cudaStream_t stream) {
    PagesParams g;
    memset(&g, 0, sizeof g);
    g.seq_lens = bt->seq_lens;
    g.block_table = bt->block_table;
    g.codes = static_cast<const uint8_t*>(at->kv_cache);
    g.scale = at->kv_scale;
    g.rows = static_cast<uint16_t*>(rows);
    g.page_scale = page_scale;
    g.B = bt->batch;
    g.max_blocks = bt->max_blocks_per_seq;
    g.num_blocks = bt->num_blocks;
    g.pages = (int32_t)pages;
    kv_fp8_pages_kernel<<<(unsigned)(pages * bt->batch), kPagesThreads, 0, stream>>>(g);
    if (cudaError_t e = cudaGetLastError()) return fail(DSA_ERR_CUDA, "latent copy launch", e);
    return DSA_OK;
}

dsa_status copy_fp16_queries(const void* q, int64_t nrows, void* out, float* factor, cudaStream_t stream) {
    const int64_t blocks = (nrows + kQueryThreads / 8 - 1) / (kQueryThreads / 8);
    q_fp16_kernel<<<(unsigned)blocks, kQueryThreads, 0, stream>>>(static_cast<const uint16_t*>(q), nrows,
                                                                  static_cast<uint16_t*>(out), factor);
    if (cudaError_t e = cudaGetLastError()) return fail(DSA_ERR_CUDA, "query copy launch", e);
    return DSA_OK;
}

bool rows_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, uint64_t rows, uint64_t row, uint32_t box_rows,
              uint32_t box_chunks) {
    const uint64_t dims[3] = {64, rows, row / 64};
    const uint64_t strides[2] = {row * 2, 128};
    const uint32_t box[3] = {64, box_rows, box_chunks};
    return make_map(map, type, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace host
}  // namespace dsa
