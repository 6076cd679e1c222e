// chunk.cu -- host side of dsa_chunk_attn (include/dsa.h): argument checks, the
// scratch layout, TMA descriptors and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/dsa.h"
#include "chunk.cuh"
#include "common.h"
#include "host.h"

using namespace dsa;
using namespace dsa::host;

namespace {

// An FP8 cache is copied as fp16 once per call, rather than converted in the kernel, when a
// sequence can have this many tiles and the copy is no larger than kCopyBytes, which bounds the
// scratch that a call needs beside its cache.  (Us, copy / kernel, 128 heads: one sequence of 16K
// positions with 16 new tokens 177 / 178, 64 456 / 572, 512 2857 / 4132, 2048 10894 / 15592; 8 sequences of
// 16K to 131K, whose copy is 1.2 GB, 64 tokens 17864 / 16706, 2 tokens 899 / 548.  One sequence
// past the bound: 2048 tokens over 48K positions 36.0 / 44.1 ms, 64K 48.5 / 58.9, 128K 98.6 / 120.1; over
// 64K 512 tokens 12.8 / 14.9, 256 6.7 / 7.5, 64 2.0 / 2.5: there the bound costs a fifth.)
constexpr int64_t kCopyTiles = 32;
constexpr int64_t kCopyBytes = int64_t(96) << 20;

// Scratch: [headers][partial slots of the pairs][the fp16 copy, a factor per page].
struct ChunkPlan {
    int pairs = 0;
    int64_t pages = 0;          // pages per sequence of the copy (0: none)
    size_t copy_off = 0, scale_off = 0, total = 0;
};

dsa_status plan_chunk(const dsa_batch* bt, const dsa_attn_inputs* at, const DevInfo& di, ChunkPlan& pl) {
    if (dsa_status st = check_batch(bt)) return st;
    if (dsa_status st = check_attn(at)) return st;
    // (token, head) rows are counted in 32 bits
    if ((int64_t)bt->num_tokens * at->H > INT32_MAX - ChunkCfg::ROWS) return DSA_ERR_UNSUPPORTED;
    if (di.sms <= 0) return fail(DSA_ERR_CUDA, "device query failed");
    if (di.max_smem < ChunkCfg::SMEM) return fail(DSA_ERR_UNSUPPORTED, "device shared memory per block too small");
    int pmax = di.sms / 2;
    if (pmax > ChunkCfg::MAX_PAIRS) pmax = ChunkCfg::MAX_PAIRS;
    // no more pairs than there can be blocks
    const int64_t rows = (int64_t)bt->num_tokens * at->H;
    const int64_t tiles = (rows + ChunkCfg::ROWS - 1) / ChunkCfg::ROWS +
                          (bt->batch < bt->num_tokens ? bt->batch : bt->num_tokens);
    const int64_t blocks = tiles * (((int64_t)bt->max_seq_len + ChunkCfg::BLOCK - 1) / ChunkCfg::BLOCK);
    pl.pairs = (int)(blocks < pmax ? blocks : pmax);
    pl.total = align256(ChunkCfg::HEAD_BYTES + (size_t)pmax * 4 * (size_t)ChunkCfg::PART_BYTES);
    if (at->kv_dtype == DSA_KV_FP8) {
        const int64_t most = bt->max_q_per_seq < bt->num_tokens ? bt->max_q_per_seq : bt->num_tokens;
        const int64_t pages = ((int64_t)bt->max_seq_len + kPage - 1) / kPage;
        if (most * at->H >= kCopyTiles * ChunkCfg::ROWS && pages * bt->batch <= kCopyBytes / (kPage * kCopyRow * 2)) {
            pl.pages = pages;
            pl.copy_off = pl.total;
            pl.scale_off = pl.copy_off + (size_t)pages * bt->batch * kPage * kCopyRow * 2;
            pl.total = align256(pl.scale_off + (size_t)pages * bt->batch * 4);
        }
    }
    return DSA_OK;
}

}  // namespace

extern "C" {

size_t dsa_chunk_scratch_size(const dsa_batch* batch, const dsa_attn_inputs* at) {
    ChunkPlan pl;
    return plan_chunk(batch, at, dev_info(), pl) == DSA_OK ? pl.total : 0;
}

dsa_status dsa_chunk_attn(const dsa_batch* batch, const dsa_attn_inputs* at, void* out, float* lse, void* status,
                          void* scratch, size_t scratch_bytes, void* stream) {
    ChunkPlan pl;
    const DevInfo di = dev_info();
    if (dsa_status st = plan_chunk(batch, at, di, pl)) return st;
    if (!out || !aligned16(out) || !status || (reinterpret_cast<uintptr_t>(status) & 3u)) return DSA_ERR_INVALID_ARG;
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) || scratch_bytes < pl.total) return DSA_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    ChunkParams p;
    memset(&p, 0, sizeof p);
    p.seq_lens = batch->seq_lens;
    p.cu_q = batch->cu_q;
    p.block_table = batch->block_table;
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.part = static_cast<uint8_t*>(scratch);
    p.status = static_cast<uint32_t*>(status);
    p.B = batch->batch;
    p.T = batch->num_tokens;
    p.H = at->H;
    p.max_blocks = batch->max_blocks_per_seq;
    p.num_blocks = batch->num_blocks;
    p.staged = (int32_t)pl.pages;
    const int64_t room = (pl.pages ? pl.pages : (int64_t)batch->max_blocks_per_seq) * kPage;
    p.max_len = (int32_t)(room < kMaxLen ? room : kMaxLen);
    p.tokens = p.max_tokens = INT32_MAX;
    p.scale_log2 = at->sm_scale * 1.4426950408889634f;
    const ChunkCache cache = at->kv_dtype != DSA_KV_FP8 ? kCacheBf16 : pl.pages ? kCacheCopy : kCacheFp8;
    CUtensorMap tm_q, tm_k, tm_v, tm_r;
    bool maps = rows_map(&tm_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, at->q, (uint64_t)batch->num_tokens * at->H, kDqk, 64,
                         ChunkCfg::KCH);
    if (cache == kCacheFp8) {
        p.codes = static_cast<const uint8_t*>(at->kv_cache);
        p.kv_scale = at->kv_scale;
        const uint64_t dims[2] = {(uint64_t)kDqk, (uint64_t)batch->num_blocks * kPage}, stride = kDqk;
        const uint32_t bk[2] = {128, 64}, br[2] = {64, 64}, bv[2] = {256, 32};
        auto code_map = [&](CUtensorMap* t, const uint32_t* box) {
            return make_map(t, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, at->kv_cache, dims, &stride, box, CU_TENSOR_MAP_SWIZZLE_NONE);
        };
        maps = maps && code_map(&tm_k, bk) && code_map(&tm_r, br) && code_map(&tm_v, bv);
    } else {
        const void* rows = at->kv_cache;
        uint64_t nrows = (uint64_t)batch->num_blocks * kPage;
        if (cache == kCacheCopy) {
            float* factors = reinterpret_cast<float*>(p.part + pl.scale_off);
            if (dsa_status st = copy_fp8_pages(batch, at, pl.pages, p.part + pl.copy_off, factors, s)) return st;
            p.page_scale = factors;
            rows = p.part + pl.copy_off;
            nrows = (uint64_t)pl.pages * batch->batch * kPage;
        }
        const CUtensorMapDataType type =
            cache == kCacheCopy ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        const uint64_t row = cache == kCacheCopy ? kCopyRow : kDqk;
        maps = maps && rows_map(&tm_k, type, rows, nrows, row, 64, 3) && rows_map(&tm_v, type, rows, nrows, row, 32, 4);
    }
    if (cache != kCacheFp8) tm_r = tm_k;         // not used
    if (!maps)
        return fail(DSA_ERR_CUDA, "tensor map encoding failed");
    const auto kernel = cache == kCacheFp8    ? &chunk_attn_kernel<kCacheFp8>
                        : cache == kCacheCopy ? &chunk_attn_kernel<kCacheCopy>
                                              : &chunk_attn_kernel<kCacheBf16>;
    if (cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(kernel), ChunkCfg::SMEM))
        return fail(DSA_ERR_CUDA, "shared memory attribute", e);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(2 * pl.pairs, 1, 1);
    cfg.blockDim = dim3(32 * ChunkCfg::warps(cache == kCacheFp8), 1, 1);
    cfg.dynamicSmemBytes = ChunkCfg::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, tm_q, tm_k, tm_v, tm_r))
        return fail(DSA_ERR_CUDA, "attention launch", e);
    if (pl.pairs < 2) return DSA_OK;
    cudaLaunchConfig_t ccfg;
    memset(&ccfg, 0, sizeof ccfg);
    ccfg.gridDim = dim3(di.sms, 1, 1);
    ccfg.blockDim = dim3(ChunkCfg::COMBINE_THREADS, 1, 1);
    ccfg.stream = s;
    ccfg.attrs = attr;
    ccfg.numAttrs = 1;
    if (cudaError_t e = cudaLaunchKernelEx(&ccfg, &chunk_combine_kernel, p, pl.pairs)) return fail(DSA_ERR_CUDA, "merge launch", e);
    return DSA_OK;
}

}  // extern "C"
