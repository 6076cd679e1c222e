// evict.cu -- host side of dsa_cache_evict (include/dsa.h): argument checks, scratch
// and launches.
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/dsa.h"
#include "common.h"
#include "evict.cuh"
#include "host.h"

using namespace dsa;
using namespace dsa::host;

namespace {

// Largest power of two up to 16 that divides both addresses and the row.
int copy_width(const dsa_cache_array& a) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.src) | reinterpret_cast<uintptr_t>(a.dst) | (uintptr_t)a.row_bytes;
    int w = 16;
    while (bits & (uintptr_t)(w - 1)) w >>= 1;
    return w;
}

dsa_status check_evict(const dsa_batch* bt, const dsa_evict_inputs* in, const int32_t* idx, const int32_t* len,
                       const void* status) {
    if (dsa_status st = check_batch(bt)) return st;
    if (!in || !in->weight || !in->new_table || !idx || !len || !status || (reinterpret_cast<uintptr_t>(status) & 3u))
        return DSA_ERR_INVALID_ARG;
    if (in->weight_stride < bt->max_seq_len || in->keep < 1 || in->sink < 0 || in->recent < 0 ||
        (int64_t)in->sink + in->recent > in->keep)
        return DSA_ERR_INVALID_ARG;
    const int64_t most = bt->max_seq_len < in->keep ? bt->max_seq_len : in->keep;   // rows a sequence can keep
    if (in->new_max_blocks < 1 || in->new_num_blocks < 1 || (int64_t)in->new_max_blocks * kPage < most) return DSA_ERR_INVALID_ARG;
    if (in->new_weight && in->new_weight_stride < most) return DSA_ERR_INVALID_ARG;
    if (in->new_weight) {
        // [first row .. last row's end) of both: new weights are written while others are read
        const float *w1 = in->weight + (int64_t)(bt->batch - 1) * in->weight_stride + bt->max_seq_len;
        const float *n1 = in->new_weight + (int64_t)(bt->batch - 1) * in->new_weight_stride + most;
        if (in->new_weight < w1 && in->weight < n1) return DSA_ERR_INVALID_ARG;
    }
    if (in->n_arrays < 0 || (in->n_arrays > 0 && !in->arrays)) return DSA_ERR_INVALID_ARG;
    if (in->n_arrays > kEvictMaxArrays || bt->batch > 65535) return DSA_ERR_UNSUPPORTED;
    for (int i = 0; i < in->n_arrays; ++i) {
        const dsa_cache_array& a = in->arrays[i];
        if (!a.src || !a.dst || a.row_bytes < 1) return DSA_ERR_INVALID_ARG;
        if (a.row_bytes / copy_width(a) > 2047) return DSA_ERR_UNSUPPORTED;   // the copy counts 32 rows' pieces in 16 bits
    }
    return DSA_OK;
}

}  // namespace

namespace {

// CTAs per sequence of the wide kernel (0: the cluster kernel serves): at least kEvictWideRange
// positions each, and all sequences at once where there are enough SMs.
int wide_ctas(const dsa_batch* bt, const DevInfo& di) {
    if (bt->max_seq_len < kEvictWide) return 0;
    const int by_len = (int)(((int64_t)bt->max_seq_len + kEvictWideRange - 1) / kEvictWideRange);
    const int by_sms = di.sms / bt->batch > 8 ? di.sms / bt->batch : di.sms < 8 ? di.sms : 8;
    return by_len < by_sms ? by_len : by_sms;
}

}  // namespace

extern "C" {

size_t dsa_evict_scratch_size(const dsa_batch* batch) {
    if (check_batch(batch) != DSA_OK) return 0;
    const DevInfo di = dev_info();
    if (di.sms <= 0) return 0;
    return 256 + align256(((size_t)di.sms + (size_t)batch->batch * (3 * kEvictBins + 2 * (size_t)wide_ctas(batch, di))) * 4);
}

dsa_status dsa_cache_evict(const dsa_batch* batch, const dsa_evict_inputs* in, int32_t* out_idx, int32_t* out_len, void* status,
                           void* scratch, size_t scratch_bytes, void* stream) {
    if (dsa_status st = check_evict(batch, in, out_idx, out_len, status)) return st;
    if (!scratch || (reinterpret_cast<uintptr_t>(scratch) & 255u) || scratch_bytes < dsa_evict_scratch_size(batch))
        return DSA_ERR_WORKSPACE;
    const DevInfo di = dev_info();
    if (di.sms <= 0) return fail(DSA_ERR_CUDA, "device query failed");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    EvictParams p;
    memset(&p, 0, sizeof p);
    p.seq_lens = batch->seq_lens;
    p.block_table = batch->block_table;
    p.new_table = in->new_table;
    p.weight = in->weight;
    p.new_weight = in->new_weight;
    p.idx = out_idx;
    p.len = out_len;
    p.status = static_cast<uint32_t*>(status);
    p.stride = in->weight_stride;
    p.new_stride = in->new_weight_stride;
    p.B = batch->batch;
    p.max_blocks = batch->max_blocks_per_seq;
    p.num_blocks = batch->num_blocks;
    p.max_len = (int32_t)(batch->max_seq_len < kMaxLen ? batch->max_seq_len : kMaxLen);
    p.new_max_blocks = in->new_max_blocks;
    p.new_num_blocks = in->new_num_blocks;
    p.keep = in->keep;
    p.sink = in->sink;
    p.recent = in->recent;
    p.n_arrays = in->n_arrays;
    for (int i = 0; i < in->n_arrays; ++i) {
        const dsa_cache_array& a = in->arrays[i];
        EvictArray& e = p.arrays[i];
        e.src = static_cast<const uint8_t*>(a.src);
        e.dst = static_cast<uint8_t*>(a.dst);
        e.bytes = a.row_bytes;
        e.width = copy_width(a);
        e.pieces = (int32_t)(a.row_bytes / e.width);
        e.magic = (uint32_t)(((uint64_t(1) << 32) + e.pieces - 1) / e.pieces);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof cfg);
    cfg.blockDim = dim3(kEvictThreads, 1, 1);
    cfg.stream = s;
    cfg.attrs = attr;
    p.ctas = wide_ctas(batch, di);
    if (p.ctas) {
        const int groups = di.sms / p.ctas < p.B ? di.sms / p.ctas : p.B;
        p.barriers = static_cast<uint32_t*>(scratch);
        p.hist = p.barriers + di.sms;
        p.counts = p.hist + (size_t)p.B * 3 * kEvictBins;
        if (cudaError_t e = cudaMemsetAsync(scratch, 0, ((size_t)di.sms + (size_t)p.B * 3 * kEvictBins) * 4, s))
            return fail(DSA_ERR_CUDA, "eviction histogram clear", e);
        cudaLaunchAttribute together;                    // the CTAs of a group wait for one another
        together.id = cudaLaunchAttributeCooperative;
        together.val.cooperative = 1;
        cfg.gridDim = dim3((unsigned)(groups * p.ctas), 1, 1);
        cfg.attrs = &together;
        cfg.numAttrs = 1;
        if (cudaError_t e = cudaLaunchKernelEx(&cfg, &evict_wide_kernel, p)) return fail(DSA_ERR_CUDA, "eviction choice launch", e);
        cfg.attrs = attr;
    } else {
        p.cluster = 1;
        while (p.cluster < 8 && (int64_t)p.cluster * 8192 < batch->max_seq_len) p.cluster *= 2;
        p.cache = (batch->max_seq_len + p.cluster - 1) / p.cluster;
        const int smem = (int)sizeof(EvictShared) + p.cache * 4;
        if (di.max_smem < smem) return fail(DSA_ERR_UNSUPPORTED, "device shared memory per block too small");
        if (cudaError_t e = set_smem_attr(reinterpret_cast<const void*>(&evict_select_kernel), (int)sizeof(EvictShared) + 8192 * 4))
            return fail(DSA_ERR_CUDA, "shared memory attribute", e);
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)p.cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(p.B * p.cluster), 1, 1);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.numAttrs = 2;
        if (cudaError_t e = cudaLaunchKernelEx(&cfg, &evict_select_kernel, p)) return fail(DSA_ERR_CUDA, "eviction choice launch", e);
    }
    if (p.n_arrays == 0 && !p.new_weight) return DSA_OK;
    const int64_t most = batch->max_seq_len < in->keep ? batch->max_seq_len : in->keep;
    cfg.gridDim = dim3((unsigned)((most + kEvictCopyRows - 1) / kEvictCopyRows), (unsigned)p.B, 1);
    cfg.blockDim = dim3(kEvictCopyThreads, 1, 1);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    if (cudaError_t e = cudaLaunchKernelEx(&cfg, &evict_copy_kernel, p)) return fail(DSA_ERR_CUDA, "eviction copy launch", e);
    return DSA_OK;
}

}  // extern "C"
