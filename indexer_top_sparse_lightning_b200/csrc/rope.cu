// rope.cu -- host side of dsa_qk_norm_rope (include/dsa.h): argument checks,
// the split of the rows over blocks, the launch.
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/dsa.h"
#include "common.h"
#include "host.h"
#include "rope.cuh"

using namespace dsa;
using namespace dsa::host;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

dsa_status check_rope(const dsa_batch* bt, const dsa_rope_inputs* in, const void* q_out, const void* k_cache,
                      const float* k_scale, const void* status) {
    if (!bt || bt->batch < 1 || bt->num_tokens < 1 || !bt->seq_lens || !bt->cu_q) return DSA_ERR_INVALID_ARG;
    if (!in || (!in->q && !in->k)) return DSA_ERR_INVALID_ARG;
    if (in->D < 8 || in->D > kRopeMaxDim || in->D % 8) return DSA_ERR_UNSUPPORTED;
    if (in->rope_dim < 0 || in->rope_dim % 16 || in->rope_off < 0 || in->rope_off % 8) return DSA_ERR_UNSUPPORTED;
    if ((int64_t)in->rope_off + in->rope_dim > in->D) return DSA_ERR_INVALID_ARG;
    if (in->rope_dim > 0 && !in->inv_freq) return DSA_ERR_INVALID_ARG;
    if (!(in->eps >= 0.0f)) return DSA_ERR_INVALID_ARG;
    auto norm_ok = [&](int32_t n, const float* g) {
        return n >= 0 && n <= in->D && n % 8 == 0 && (n == 0 || (g && aligned(g, 16)));
    };
    if (in->q) {
        if (in->H < 1 || !q_out || !aligned(in->q, 16) || !aligned(q_out, 16)) return DSA_ERR_INVALID_ARG;
        if (in->q_stride_t % 8 || in->q_stride_h % 8 || in->q_stride_t < 0 || in->q_stride_h < 0)
            return DSA_ERR_INVALID_ARG;
        if (!norm_ok(in->q_norm, in->q_gamma)) return DSA_ERR_INVALID_ARG;
        // rows written over the queries must be the very rows that were read
        if (q_out == in->q && (in->q_stride_h != in->D || in->q_stride_t != (int64_t)in->H * in->D))
            return DSA_ERR_INVALID_ARG;
    }
    if (in->k) {
        if (!bt->block_table || bt->max_blocks_per_seq < 1 || bt->num_blocks < 1) return DSA_ERR_INVALID_ARG;
        if (!k_cache || !status || !aligned(status, 4) || !aligned(in->k, 16) || !aligned(k_cache, 16)) return DSA_ERR_INVALID_ARG;
        if (in->k_stride_t % 8 || in->k_stride_t < 0) return DSA_ERR_INVALID_ARG;
        if (!norm_ok(in->k_norm, in->k_gamma)) return DSA_ERR_INVALID_ARG;
        if (in->kv_dtype != DSA_KV_BF16 && in->kv_dtype != DSA_KV_FP8) return DSA_ERR_INVALID_ARG;
        if (in->kv_dtype == DSA_KV_FP8) {
            if (!k_scale || !aligned(k_scale, 4)) return DSA_ERR_INVALID_ARG;
            if (in->D != kDqk) return DSA_ERR_UNSUPPORTED;
        }
    }
    return DSA_OK;
}

template <int NV>
cudaError_t launch(const RopeParams& p, int64_t blocks, cudaStream_t s) {
    // (the kernel waits for the one before it ahead of its first read)
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.gridDim = dim3((unsigned)blocks, 1, 1);
    cfg.blockDim = dim3(kRopeThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, &qk_norm_rope_kernel<NV>, p);
}

}  // namespace

extern "C" dsa_status dsa_qk_norm_rope(const dsa_batch* batch, const dsa_rope_inputs* in, void* q_out, void* k_cache,
                                       float* k_scale, void* status, void* stream) {
    if (dsa_status st = check_rope(batch, in, q_out, k_cache, k_scale, status)) return st;
    const DevInfo di = dev_info();
    if (di.sms <= 0) return fail(DSA_ERR_CUDA, "device query failed");
    RopeParams p;
    memset(&p, 0, sizeof p);
    p.seq_lens = batch->seq_lens;
    p.cu_q = batch->cu_q;
    p.block_table = batch->block_table;
    p.positions = in->positions;
    p.q = static_cast<const uint16_t*>(in->q);
    p.k = static_cast<const uint16_t*>(in->k);
    p.q_stride_t = in->q_stride_t;
    p.q_stride_h = in->q_stride_h;
    p.k_stride_t = in->k_stride_t;
    p.q_gamma = in->q_gamma;
    p.k_gamma = in->k_gamma;
    p.inv_freq = in->inv_freq;
    p.q_out = static_cast<uint16_t*>(q_out);
    p.k_cache = k_cache;
    p.k_scale = k_scale;
    p.status = static_cast<uint32_t*>(status);
    p.B = batch->batch;
    p.T = batch->num_tokens;
    p.H = in->H;
    p.D = in->D;
    p.max_blocks = batch->max_blocks_per_seq;
    p.num_blocks = batch->num_blocks;
    p.q_norm = in->q_norm;
    p.k_norm = in->k_norm;
    p.r0 = in->rope_off;
    p.R = in->rope_dim;
    p.interleaved = in->interleaved ? 1 : 0;
    p.fp8 = in->kv_dtype == DSA_KV_FP8 ? 1 : 0;
    p.eps = in->eps;
    // tokens whose angle tables fit a block
    const int by_table = p.R > 0 ? kRopeTable / (p.R / 2) : kRopeGroups;
    const int tmax = by_table < kRopeGroups ? by_table : kRopeGroups;
    int64_t blocks = 0;
    if (in->q) {
        if (p.H < kRopeGroups) {
            // several tokens share a block so that its row slots are filled
            p.tpc = kRopeGroups / p.H < tmax ? kRopeGroups / p.H : tmax;
            p.hpc = p.H;
        } else {
            // one token: as many of its heads as still leave two blocks per SM (a block's start, places
            // and angles, serves more rows), at least one row per slot.  (With eight per SM 1000 ragged
            // tokens of 64 heads of 128 took 14.5 us for 13.4, 415 of 128 heads of 576 37 for 32.)
            const int64_t slots = (int64_t)p.T * (((int64_t)p.H + kRopeGroups - 1) / kRopeGroups);
            const int64_t rounds = slots / ((int64_t)di.sms * 2);
            p.tpc = 1;
            const int64_t hpc = (int64_t)kRopeGroups * (rounds < 1 ? 1 : rounds);
            p.hpc = hpc < p.H ? (int)hpc : p.H;
        }
        p.hsplit = (int)(((int64_t)p.H + p.hpc - 1) / p.hpc);
        blocks = ((int64_t)p.T + p.tpc - 1) / p.tpc * p.hsplit;
    } else {
        p.tpc = p.hpc = p.hsplit = 1;
    }
    if (blocks > INT32_MAX) return DSA_ERR_UNSUPPORTED;
    p.q_blocks = (int32_t)blocks;
    if (in->k) {
        // few tokens: one per block, so that no key waits for the angles of another
        p.ktpc = p.T <= di.sms ? 1 : tmax;
        blocks += ((int64_t)p.T + p.ktpc - 1) / p.ktpc;
    } else {
        p.ktpc = 1;
    }
    if (blocks > INT32_MAX) return DSA_ERR_UNSUPPORTED;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    // rounds of 64 elements per row, the next instantiated count
    const int nv = (p.D + 63) / 64;
    const cudaError_t e = nv <= 1 ? launch<1>(p, blocks, s)
                        : nv <= 2 ? launch<2>(p, blocks, s)
                        : nv <= 4 ? launch<4>(p, blocks, s)
                        : nv <= 8 ? launch<8>(p, blocks, s)
                        : nv <= 9 ? launch<9>(p, blocks, s)
                                  : launch<16>(p, blocks, s);
    if (e) return fail(DSA_ERR_CUDA, "norm and rotation launch", e);
    return DSA_OK;
}
