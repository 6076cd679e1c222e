// weight.cu -- host side of dsa_attn_weight (include/dsa.h): argument checks, the
// scratch layout, the windows of new tokens, the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/dsa.h"
#include "common.h"
#include "host.h"
#include "weight.cuh"

using namespace dsa;
using namespace dsa::host;

namespace {

// Sums per tile are kept for windows of new tokens whose sums fit this many bytes (a window
// has one tile per sequence at least).
constexpr int64_t kPartBytes = int64_t(256) << 20;

// Scratch: [sums per tile][FP8: the sequences' rows as fp16, a factor per page; the queries as
// fp16, a factor per row].
struct WeightPlan {
    int nr = 128;               // rows of a tile
    bool direct = true;         // every sequence has one tile: sums are added in place
    int64_t window = 0;         // new tokens per sequence and pass
    int64_t tiles = 1;          // tiles per sequence and pass
    int64_t part_stride = 0;
    int64_t pages = 0;
    size_t copy_off = 0, scale_off = 0, q_off = 0, factor_off = 0, total = 0;
};

dsa_status plan_weight(const dsa_batch* bt, const dsa_attn_inputs* at, const DevInfo& di, WeightPlan& pl) {
    if (dsa_status st = check_batch(bt)) return st;
    if (dsa_status st = check_attn(at)) return st;
    const int64_t T = bt->num_tokens, H = at->H;
    if (T * H > INT32_MAX - 256) return DSA_ERR_UNSUPPORTED;     // (token, head) rows are counted in 32 bits
    if (di.sms <= 0) return fail(DSA_ERR_CUDA, "device query failed");
    if (di.max_smem < WeightCfg<128>::SMEM || di.max_smem < WeightCfg<256>::SMEM)
        return fail(DSA_ERR_UNSUPPORTED, "device shared memory per block too small");
    const int64_t nq = bt->max_q_per_seq < T ? bt->max_q_per_seq : T;
    pl.nr = nq * H <= 128 ? 128 : 256;
    pl.direct = nq * H <= pl.nr;
    pl.window = nq;
    size_t off = 0;
    if (!pl.direct) {
        pl.part_stride = ((int64_t)bt->max_seq_len + 255) / 256 * 256;
        const int64_t per_tile = pl.part_stride * 4 * bt->batch;
        int64_t tiles = kPartBytes / per_tile;
        if (tiles < 1) tiles = 1;
        pl.tiles = (nq * H + pl.nr - 1) / pl.nr;
        if (pl.tiles > tiles) {
            // whole tokens whose rows fill at most `tiles` tiles (H <= 128 rows: at least two fit)
            pl.window = tiles * pl.nr / H;
            pl.tiles = (pl.window * H + pl.nr - 1) / pl.nr;
        }
        off = align256((size_t)(pl.tiles * per_tile));
    }
    if (bt->batch > 65535) return DSA_ERR_UNSUPPORTED;           // the sums' grid
    if (at->kv_dtype == DSA_KV_FP8) {
        pl.pages = ((int64_t)bt->max_seq_len + kPage - 1) / kPage;
        if (pl.pages * bt->batch > INT32_MAX / kPage) return DSA_ERR_UNSUPPORTED;   // rows of the copy, in 32 bits
        pl.copy_off = off;
        pl.scale_off = off + (size_t)pl.pages * bt->batch * kPage * kCopyRow * 2;
        pl.q_off = align256(pl.scale_off + (size_t)pl.pages * bt->batch * 4);
        pl.factor_off = align256(pl.q_off + (size_t)(T * H) * kDqk * 2);
        off = pl.factor_off + (size_t)(T * H) * 4;
    }
    pl.total = align256(off + 1);                                // never 0
    return DSA_OK;
}

template <int NR>
dsa_status launch(WeightParams& p, const WeightPlan& pl, const CUtensorMap& tm_q, const CUtensorMap& tm_k, const DevInfo& di,
                  int64_t max_seq_len, cudaStream_t s) {
    using Cfg = WeightCfg<NR>;
    const auto kernel = pl.pages ? &attn_weight_kernel<NR, true> : &attn_weight_kernel<NR, false>;
    if (cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(kernel), Cfg::SMEM))
        return fail(DSA_ERR_CUDA, "shared memory attribute", e);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    // no more pairs than there can be blocks
    const int64_t blocks = (int64_t)p.B * pl.tiles * ((max_seq_len + Cfg::BLOCK - 1) / Cfg::BLOCK);
    const int pairs = (int)(blocks < di.sms / 2 ? blocks : di.sms / 2);
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3(2 * pairs, 1, 1);
    cfg.blockDim = dim3(Cfg::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cfg::SMEM;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, tm_q, tm_k)) return fail(DSA_ERR_CUDA, "attention weight launch", e);
    if (pl.direct) return DSA_OK;
    cfg.gridDim = dim3((unsigned)((max_seq_len + kWeightSumThreads - 1) / kWeightSumThreads), (unsigned)p.B, 1);
    cfg.blockDim = dim3(kWeightSumThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, &weight_sum_kernel<NR>, p)) return fail(DSA_ERR_CUDA, "weight sum launch", e);
    return DSA_OK;
}

}  // namespace

extern "C" {

size_t dsa_weight_scratch_size(const dsa_batch* batch, const dsa_attn_inputs* at) {
    WeightPlan pl;
    return plan_weight(batch, at, dev_info(), pl) == DSA_OK ? pl.total : 0;
}

dsa_status dsa_attn_weight(const dsa_batch* batch, const dsa_attn_inputs* at, const float* lse, float* weight, int64_t stride,
                           float decay, void* status, void* scratch, size_t scratch_bytes, void* stream) {
    WeightPlan pl;
    const DevInfo di = dev_info();
    if (dsa_status st = plan_weight(batch, at, di, pl)) return st;
    if (!lse || !weight || !status || (reinterpret_cast<uintptr_t>(status) & 3u) || stride < batch->max_seq_len)
        return DSA_ERR_INVALID_ARG;
    if (!(decay >= 0.0f) || decay > 3.4e38f) return DSA_ERR_INVALID_ARG;
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) || scratch_bytes < pl.total) return DSA_ERR_WORKSPACE;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    uint8_t* sc = static_cast<uint8_t*>(scratch);
    WeightParams p;
    memset(&p, 0, sizeof p);
    p.seq_lens = batch->seq_lens;
    p.cu_q = batch->cu_q;
    p.block_table = batch->block_table;
    p.B = batch->batch;
    p.T = batch->num_tokens;
    p.H = at->H;
    p.max_blocks = batch->max_blocks_per_seq;
    p.num_blocks = batch->num_blocks;
    p.staged = (int32_t)pl.pages;
    p.max_len = (int32_t)(batch->max_seq_len < kMaxLen ? batch->max_seq_len : kMaxLen);
    p.max_tokens = batch->max_q_per_seq;
    p.lse = lse;
    p.weight = weight;
    p.part = pl.direct ? nullptr : reinterpret_cast<float*>(sc);
    p.stride = stride;
    p.part_stride = pl.part_stride;
    p.tiles_per_seq = (int32_t)pl.tiles;
    p.status = static_cast<uint32_t*>(status);
    p.scale_log2 = at->sm_scale * 1.4426950408889634f;
    const void *q = at->q, *rows = at->kv_cache;
    uint64_t nrows = (uint64_t)batch->num_blocks * kPage;
    const int64_t qrows = (int64_t)batch->num_tokens * at->H;
    if (pl.pages) {
        float* page_scale = reinterpret_cast<float*>(sc + pl.scale_off);
        float* factor = reinterpret_cast<float*>(sc + pl.factor_off);
        if (dsa_status st = copy_fp8_pages(batch, at, pl.pages, sc + pl.copy_off, page_scale, s)) return st;
        if (dsa_status st = copy_fp16_queries(at->q, qrows, sc + pl.q_off, factor, s)) return st;
        p.page_scale = page_scale;
        p.q_factor = factor;
        q = sc + pl.q_off;
        rows = sc + pl.copy_off;
        nrows = (uint64_t)pl.pages * batch->batch * kPage;
    }
    const CUtensorMapDataType type = pl.pages ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    CUtensorMap tm_q, tm_k;
    if (!rows_map(&tm_q, type, q, (uint64_t)qrows, kDqk, (uint32_t)pl.nr / 2, 9) ||
        !rows_map(&tm_k, type, rows, nrows, pl.pages ? kCopyRow : kDqk, 64, 1))
        return fail(DSA_ERR_CUDA, "tensor map encoding failed");
    // windows of new tokens, each added on top of the one before
    const int64_t nq = batch->max_q_per_seq < batch->num_tokens ? batch->max_q_per_seq : batch->num_tokens;
    for (int64_t t0 = 0; t0 < nq; t0 += pl.window) {
        p.tok0 = (int32_t)t0;
        p.tokens = (int32_t)pl.window;
        p.decay = t0 == 0 ? decay : 1.0f;
        if (dsa_status st = pl.nr == 128 ? launch<128>(p, pl, tm_q, tm_k, di, batch->max_seq_len, s)
                                         : launch<256>(p, pl, tm_q, tm_k, di, batch->max_seq_len, s))
            return st;
    }
    return DSA_OK;
}

}  // extern "C"
