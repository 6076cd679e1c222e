// evict.cuh -- eviction from the paged caches by accumulated attention weight.
//
// Of a sequence's L cached positions, `keep` stay: the first `sink`, the last
// `recent`, and the others by (weight descending, position ascending).  The
// kept positions are listed in ascending order, and their rows are copied, in
// that order, to the sequence's new pages: position idx[j] becomes position j.
//
// evict_select_kernel: a cluster of CTAs per sequence (one per ~8192 positions,
// at most eight), each on a contiguous range.  The keep-th largest key is found by
// three digit histograms (11, 11 and 10 bits of the order-preserving key), each
// joined over the cluster through distributed shared memory; then the keys above
// it, and as many equal to it as are wanted, lowest positions first, are written
// with counts and ballots in position order.  A range's keys stay in shared
// memory.  Weights of zero (positions nobody attends to) are
// common: they are counted with ballots, since a histogram bin that a whole warp
// adds to takes its lanes one by one.
//
// Longer sequences (kEvictWide positions and more) take the same steps with a group of up to
// all SMs' CTAs each (evict_wide_kernel), joined through histograms and counts in
// scratch; a range's keys stay in shared memory where they fit: eight CTAs would need 270 us for a million positions, most of it histogram
// adds, which a CTA takes one by one.
//
// evict_copy_kernel: memory-bound, every kept row read and written once.  A block
// takes 32 rows: their places are resolved once, then each array's rows are copied
// in 16-byte pieces (or what their width allows), four loads in flight per thread.
// (Blocks that stay and resolve the next rows' places while they copy were slower, 185 for
// 147 us below.)
//
// Measured: 32 sequences of 28K to 32K cut to 8192 positions, latent rows and index keys,
// 147 us: 24 to choose, 122 to copy 740 MB (6.07 TB/s).  A million positions cut to 65536, FP8 rows:
// 55 us, about half each for the choice and the copy.
#pragma once
#include "common.h"
#include "paging.cuh"
#include "ptx.cuh"

namespace dsa {

constexpr int kEvictThreads = 1024;
constexpr int kEvictWarps = kEvictThreads / 32;   // a warp's lanes
static_assert(kEvictWarps == 32, "one lane per warp in the sums over warps");
constexpr int kEvictBins = 2048;
constexpr int kEvictWide = 65537;           // longest sequence from which the wide kernels are used
constexpr int kEvictWideRange = 4096;       // positions per CTA there, at least
constexpr int kEvictWideKeys = 9216;        // keys of a CTA there that shared memory holds
constexpr int kEvictMaxArrays = 8;
constexpr int kEvictCopyThreads = 256;
constexpr int kEvictCopyRows = 32;

struct EvictArray {
    const uint8_t* src;       // rows of `bytes` bytes
    uint8_t* dst;
    int64_t bytes;
    int32_t width;            // bytes moved at a time (a power of two up to 16)
    int32_t pieces;           // bytes / width
    uint32_t magic;           // 2^32 / pieces, rounded up
};

struct EvictParams {
    const int32_t* seq_lens;
    const int32_t* block_table;
    const int32_t* new_table;
    const float* weight;      // [B, stride]
    float* new_weight;        // [B, new_stride] or null
    int32_t* idx;             // [B, keep]
    int32_t* len;             // [B]
    uint32_t* status;
    int64_t stride, new_stride;
    int32_t B, max_blocks, num_blocks, max_len;
    int32_t new_max_blocks, new_num_blocks;
    int32_t keep, sink, recent;
    int32_t cluster;          // CTAs per sequence
    int32_t cache;            // keys of a CTA's range at most (in shared memory)
    int32_t n_arrays;
    // the wide kernel: CTAs per group; a barrier count per group and [B][3][2048] digit counts
    // (zero at first), then [B][ctas][2] counts of keys above and equal
    int32_t ctas;
    uint32_t* barriers;
    uint32_t* hist;
    uint32_t* counts;
    EvictArray arrays[kEvictMaxArrays];
};

struct EvictShared {
    uint32_t hist[kEvictBins];
    uint32_t warp_sum[kEvictWarps];
    uint32_t warp_gt[kEvictWarps], warp_eq[kEvictWarps];
    uint32_t cta_gt, cta_eq;  // of this CTA's range
    uint32_t digit, above;    // result of a digit's search
    uint32_t gt_before, eq_before;
    int arrived;              // the group's barrier was passed
};

__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* local, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}

// Sum of the entries of the warps before this one.
__device__ __forceinline__ uint32_t sum_before(const uint32_t* per_warp) {
    const uint32_t lane = threadIdx.x & 31;
    return __reduce_add_sync(0xffffffffu, lane < threadIdx.x >> 5 ? per_warp[lane] : 0u);
}
// ... of all warps.
__device__ __forceinline__ uint32_t sum_all(const uint32_t* per_warp) {
    return __reduce_add_sync(0xffffffffu, per_warp[threadIdx.x & 31]);
}

// Length of sequence b as the kernels use it; out-of-range lengths are cut (and reported).
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
    const int L = __ldg(p.seq_lens + b);
    if (L > p.max_len || L < 0) {
        if (threadIdx.x == 0) atomicCAS(p.status, 0u, (uint32_t)kStBounds);
        return L < 0 ? 0 : p.max_len;
    }
    return L;
}

// Writes the positions that stay of this warp's range [w0, w1), in order, behind those of
// the warps and CTAs before.
template <typename Key>
__device__ __forceinline__ void evict_emit(const EvictShared* s, int32_t* out, int lo, int w0, int w1, uint32_t prefix,
                                           uint32_t need, Key key_at) {
    constexpr int BATCH = 8;
    const int lane = threadIdx.x & 31;
    const uint32_t g = s->gt_before + sum_before(s->warp_gt);
    uint32_t e = s->eq_before + sum_before(s->warp_eq);
    uint32_t at = g + (e < need ? e : need);
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32 * BATCH) {
        uint32_t k[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int i = i0 + 32 * u + lane;
            k[u] = i < w1 ? key_at(i) : 0u;
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int i = i0 + 32 * u + lane;
            const bool in = i < w1;
            const uint32_t me = __ballot_sync(0xffffffffu, in && k[u] == prefix);
            const bool sel = in && (k[u] > prefix || (k[u] == prefix && e + __popc(me & below) < need));
            const uint32_t ms = __ballot_sync(0xffffffffu, sel);
            if (sel) out[at + __popc(ms & below)] = lo + i;
            at += __popc(ms);
            e += __popc(me);
        }
    }
}

__global__ void __launch_bounds__(kEvictThreads, 1) evict_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ uint8_t raw[];
    EvictShared* s = reinterpret_cast<EvictShared*>(raw);
    uint32_t* s_key = reinterpret_cast<uint32_t*>(raw + sizeof(EvictShared));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int b = (int)blockIdx.x / p.cluster;
    griddep_launch_dependents();
    griddep_wait();
    const int L = evict_len(p, b), keep = p.keep;
    int32_t* out = p.idx + (int64_t)b * keep;
    if (rank == 0 && threadIdx.x == 0) p.len[b] = L < keep ? L : keep;
    if (L <= keep) {
        // everything stays (every CTA of the cluster leaves here)
        for (int64_t i = (int64_t)rank * kEvictThreads + threadIdx.x; i < keep; i += (int64_t)p.cluster * kEvictThreads)
            out[i] = i < L ? (int32_t)i : -1;
        return;
    }
    const int per = (L + p.cluster - 1) / p.cluster;
    const int64_t lo64 = (int64_t)per * rank;
    const int lo = lo64 < L ? (int)lo64 : L;
    const int n = L - lo < per ? L - lo : per;           // this CTA's positions lo .. lo + n - 1
    const float* w = p.weight + (int64_t)b * p.stride + lo;
    // Keys compare like weights; NaN lies below everything, positions that stay in any case above.
    auto make_key = [&](int i) -> uint32_t {
        const float x = __ldg(w + i);
        const int pos = lo + i;
        if (pos < p.sink || pos >= L - p.recent) return 0xFFFFFFFFu;
        return x != x ? 0u : order_key(x);
    };
    auto key_at = [&](int i) -> uint32_t { return s_key[i]; };
    constexpr uint32_t ZERO = 0x80000000u;               // order_key(0)
    constexpr int BATCH = 8;

    uint32_t prefix = 0, need = (uint32_t)keep;          // digits found; keys still wanted among those that share them
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        const uint32_t mask = pass == 2 ? 1023u : 2047u;
        const uint32_t above_mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
        for (int i = threadIdx.x; i < kEvictBins; i += kEvictThreads) s->hist[i] = 0;
        __syncthreads();
        uint32_t zeros = 0;
        for (int i0 = 0; i0 < n; i0 += kEvictThreads * BATCH) {
            uint32_t k[BATCH];
            bool in[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int i = i0 + u * kEvictThreads + (int)threadIdx.x;
                in[u] = i < n;
                k[u] = !in[u] ? 0u : pass == 0 ? make_key(i) : key_at(i);
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int i = i0 + u * kEvictThreads + (int)threadIdx.x;
                if (in[u] && pass == 0) s_key[i] = k[u];
                const bool here = in[u] && (k[u] & above_mask) == prefix;
                const uint32_t z = __ballot_sync(0xffffffffu, here && k[u] == ZERO);
                zeros += __popc(z);
                if (here && k[u] != ZERO) atomicAdd(&s->hist[(k[u] >> shift) & mask], 1u);
            }
        }
        if (lane == 0 && zeros) atomicAdd(&s->hist[(ZERO >> shift) & mask], zeros);
        cluster_sync();
        // the whole sequence's histogram, two bins a thread, highest bins first
        const int bin1 = kEvictBins - 1 - 2 * (int)threadIdx.x, bin0 = bin1 - 1;
        uint32_t c1 = 0, c0 = 0;
        for (int r = 0; r < p.cluster; ++r) {
            c1 += ld_cluster_u32(&s->hist[bin1], (uint32_t)r);
            c0 += ld_cluster_u32(&s->hist[bin0], (uint32_t)r);
        }
        uint32_t x = c1 + c0;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, d);
            if (lane >= d) x += y;
        }
        if (lane == 31) s->warp_sum[warp] = x;
        __syncthreads();
        uint32_t before = x - (c1 + c0);
        before += sum_before(s->warp_sum);
        // keys in bins above bin1: `before`; the wanted key's bin holds the need-th
        if (before < need && need <= before + c1) {
            s->digit = (uint32_t)bin1;
            s->above = before;
        } else if (before + c1 < need && need <= before + c1 + c0) {
            s->digit = (uint32_t)bin0;
            s->above = before + c1;
        }
        // every CTA has read the histograms, and its result is there, before the next pass
        cluster_sync();
        prefix |= s->digit << shift;
        need -= s->above;
    }
    // keys above `prefix` stay, and `need` of those equal to it, lowest positions first
    const int span = (n + kEvictWarps - 1) / kEvictWarps;
    const int w0 = warp * span < n ? warp * span : n, w1 = w0 + span < n ? w0 + span : n;
    uint32_t gt = 0, eq = 0;
    for (int i0 = w0; i0 < w1; i0 += 32 * BATCH) {
        uint32_t k[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const int i = i0 + 32 * u + lane;
            k[u] = i < w1 ? key_at(i) : 0u;
        }
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            const bool in = i0 + 32 * u + lane < w1;
            gt += __popc(__ballot_sync(0xffffffffu, in && k[u] > prefix));
            eq += __popc(__ballot_sync(0xffffffffu, in && k[u] == prefix));
        }
    }
    if (lane == 0) {
        s->warp_gt[warp] = gt;
        s->warp_eq[warp] = eq;
    }
    __syncthreads();
    if (warp == 0) {
        const uint32_t g = sum_all(s->warp_gt), e = sum_all(s->warp_eq);
        if (lane == 0) {
            s->cta_gt = g;
            s->cta_eq = e;
        }
    }
    cluster_sync();
    if (threadIdx.x == 0) {
        uint32_t g = 0, e = 0;
        for (uint32_t r = 0; r < rank; ++r) {
            g += ld_cluster_u32(&s->cta_gt, r);
            e += ld_cluster_u32(&s->cta_eq, r);
        }
        s->gt_before = g;
        s->eq_before = e;
    }
    cluster_sync();          // (no CTA leaves while another reads its counts)
    evict_emit(s, out, lo, w0, w1, prefix, need, key_at);
}

// Waits until all CTAs of the group have arrived `target` times in all.  False (and reported)
// after the wait limit.
__device__ __forceinline__ bool evict_group_barrier(const EvictParams& p, EvictShared* s, uint32_t* count, uint32_t target) {
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        atom_add_acq_rel_gpu(count, 1u);
        const uint32_t us = __ldcg(p.status + 1);        // test hook: wait limit in microseconds
        const uint64_t limit = us ? (uint64_t)us * 1000u : kWaitTimeoutNs, t0 = globaltimer();
        s->arrived = 1;
        while (ld_acquire_gpu(count) < target)
            if (globaltimer() - t0 > limit) {
                s->arrived = 0;
                atomicCAS(p.status, 0u, (uint32_t)kStTimeout);
                break;
            }
    }
    __syncthreads();
    return s->arrived != 0;
}

// Long sequences: a group of CTAs each, all groups at once (a cooperative launch), a group's
// sequences one after another.  The steps are those of the cluster kernel, joined through
// histograms and counts in scratch and a barrier of the group.
__global__ void __launch_bounds__(kEvictThreads, 1) evict_wide_kernel(const __grid_constant__ EvictParams p) {
    __shared__ EvictShared s_all;
    __shared__ uint32_t s_key[kEvictWideKeys];
    EvictShared* s = &s_all;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = (int)blockIdx.x / p.ctas, cta = (int)blockIdx.x % p.ctas;
    const int groups = (int)gridDim.x / p.ctas, keep = p.keep;
    constexpr uint32_t ZERO = 0x80000000u;               // order_key(0)
    constexpr int BATCH = 4;
    uint32_t* barrier = p.barriers + group;
    uint32_t arrivals = 0;
    for (int b = group; b < p.B; b += groups) {
        const int L = evict_len(p, b);
        int32_t* out = p.idx + (int64_t)b * keep;
        if (cta == 0 && threadIdx.x == 0) p.len[b] = L < keep ? L : keep;
        if (L <= keep) {
            for (int64_t i = (int64_t)cta * kEvictThreads + threadIdx.x; i < keep; i += (int64_t)p.ctas * kEvictThreads)
                out[i] = i < L ? (int32_t)i : -1;
            continue;
        }
        const int per = (L + p.ctas - 1) / p.ctas;
        const int64_t lo64 = (int64_t)per * cta;
        const int lo = lo64 < L ? (int)lo64 : L;
        const int n = L - lo < per ? L - lo : per;
        const float* w = p.weight + (int64_t)b * p.stride + lo;
        // the keys of a range that fits stay in shared memory after the first step
        const bool fits = n <= kEvictWideKeys;
        bool kept = false;
        auto key_at = [&](int i) -> uint32_t {
            if (kept) return s_key[i];
            const float x = __ldg(w + i);
            const int pos = lo + i;
            if (pos < p.sink || pos >= L - p.recent) return 0xFFFFFFFFu;
            return x != x ? 0u : order_key(x);
        };
        uint32_t prefix = 0, need = (uint32_t)keep;
#pragma unroll 1
        for (int d = 0; d < 3; ++d, kept = fits) {
            const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
            const uint32_t mask = d == 2 ? 1023u : 2047u;
            const uint32_t above_mask = d == 0 ? 0u : d == 1 ? 0xFFE00000u : 0xFFFFFC00u;
            uint32_t* hist = p.hist + ((int64_t)b * 3 + d) * kEvictBins;
            for (int i = threadIdx.x; i < kEvictBins; i += kEvictThreads) s->hist[i] = 0;
            __syncthreads();
            uint32_t zeros = 0;
            for (int i0 = 0; i0 < n; i0 += kEvictThreads * BATCH) {
                uint32_t k[BATCH];
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int i = i0 + u * kEvictThreads + (int)threadIdx.x;
                    k[u] = i < n ? key_at(i) : 0u;
                }
#pragma unroll
                for (int u = 0; u < BATCH; ++u) {
                    const int i = i0 + u * kEvictThreads + (int)threadIdx.x;
                    if (d == 0 && fits && i < n) s_key[i] = k[u];
                    const bool here = i < n && (k[u] & above_mask) == prefix;
                    zeros += __popc(__ballot_sync(0xffffffffu, here && k[u] == ZERO));
                    if (here && k[u] != ZERO) atomicAdd(&s->hist[(k[u] >> shift) & mask], 1u);
                }
            }
            if (lane == 0 && zeros) atomicAdd(&s->hist[(ZERO >> shift) & mask], zeros);
            __syncthreads();
            for (int i = threadIdx.x; i < kEvictBins; i += kEvictThreads)
                if (s->hist[i]) atomicAdd(hist + i, s->hist[i]);
            if (!evict_group_barrier(p, s, barrier, arrivals += p.ctas)) return;
            // the bin that holds the need-th key, highest bins first, two a thread
            const int bin1 = kEvictBins - 1 - 2 * (int)threadIdx.x, bin0 = bin1 - 1;
            const uint32_t c1 = __ldcg(hist + bin1), c0 = __ldcg(hist + bin0);
            uint32_t x = c1 + c0;
#pragma unroll
            for (int e = 1; e < 32; e <<= 1) {
                const uint32_t y = __shfl_up_sync(0xffffffffu, x, e);
                if (lane >= e) x += y;
            }
            if (lane == 31) s->warp_sum[warp] = x;
            __syncthreads();
            uint32_t before = x - (c1 + c0);
            before += sum_before(s->warp_sum);
            if (before < need && need <= before + c1) {
                s->digit = (uint32_t)bin1;
                s->above = before;
            } else if (before + c1 < need && need <= before + c1 + c0) {
                s->digit = (uint32_t)bin0;
                s->above = before + c1;
            }
            __syncthreads();
            prefix |= s->digit << shift;
            need -= s->above;
            __syncthreads();
        }
        // keys above `prefix` stay, and `need` of those equal to it, lowest positions first
        const int span = (n + kEvictWarps - 1) / kEvictWarps;
        const int w0 = warp * span < n ? warp * span : n, w1 = w0 + span < n ? w0 + span : n;
        uint32_t gt = 0, eq = 0;
        for (int i0 = w0; i0 < w1; i0 += 32 * BATCH) {
            uint32_t k[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const int i = i0 + 32 * u + lane;
                k[u] = i < w1 ? key_at(i) : 0u;
            }
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                const bool in = i0 + 32 * u + lane < w1;
                gt += __popc(__ballot_sync(0xffffffffu, in && k[u] > prefix));
                eq += __popc(__ballot_sync(0xffffffffu, in && k[u] == prefix));
            }
        }
        if (lane == 0) {
            s->warp_gt[warp] = gt;
            s->warp_eq[warp] = eq;
        }
        __syncthreads();
        uint32_t* counts = p.counts + 2 * (int64_t)b * p.ctas;
        const uint32_t g_all = sum_all(s->warp_gt), e_all = sum_all(s->warp_eq);
        if (threadIdx.x == 0) {
            counts[2 * cta] = g_all;
            counts[2 * cta + 1] = e_all;
        }
        if (!evict_group_barrier(p, s, barrier, arrivals += p.ctas)) return;
        // counts of the CTAs before
        if (warp == 0) {
            uint32_t g = 0, e = 0;
            for (int q = lane; q < cta; q += 32) {
                g += __ldcg(counts + 2 * q);
                e += __ldcg(counts + 2 * q + 1);
            }
            g = __reduce_add_sync(0xffffffffu, g);
            e = __reduce_add_sync(0xffffffffu, e);
            if (lane == 0) {
                s->gt_before = g;
                s->eq_before = e;
            }
        }
        __syncthreads();
        evict_emit(s, out, lo, w0, w1, prefix, need, key_at);
        __syncthreads();             // the sums are free for the next sequence
    }
}

template <typename V>
__device__ __forceinline__ void evict_copy_rows(const EvictArray& a, const int64_t* s_src, const int64_t* s_dst, int rows) {
    constexpr int U = 4;
    const int total = rows * a.pieces;
    for (int i0 = (int)threadIdx.x; i0 < total; i0 += U * kEvictCopyThreads) {
        V v[U];
        V* to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kEvictCopyThreads;
            to[u] = nullptr;
            if (i >= total) continue;
            // rows * pieces < 2^16 for the widths in use: exact (a.magic is 2^32 / pieces rounded up)
            const int r = a.pieces == 1 ? i : (int)__umulhi((uint32_t)i, a.magic);
            const int c = i - r * a.pieces;
            if (s_src[r] < 0) continue;
            v[u] = *(reinterpret_cast<const V*>(a.src + s_src[r] * a.bytes) + c);
            to[u] = reinterpret_cast<V*>(a.dst + s_dst[r] * a.bytes) + c;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (to[u]) *to[u] = v[u];
    }
}

__global__ void __launch_bounds__(kEvictCopyThreads, 6) evict_copy_kernel(const __grid_constant__ EvictParams p) {
    __shared__ int64_t s_src[kEvictCopyRows], s_dst[kEvictCopyRows];
    griddep_wait();
    const int b = (int)blockIdx.y;
    const int L = evict_len(p, b);
    const int count = L < p.keep ? L : p.keep;
    const int j0 = (int)blockIdx.x * kEvictCopyRows;
    if (j0 >= count) return;
    const int rows = count - j0 < kEvictCopyRows ? count - j0 : kEvictCopyRows;
    if ((int)threadIdx.x < rows) {
        const int j = j0 + (int)threadIdx.x;
        const int pos = __ldcg(p.idx + (int64_t)b * p.keep + j);
        int64_t src = -1, dst = -1;
        bool bad = true;
        if (pos >= 0 && pos < L) {
            if (p.n_arrays > 0) {                        // (without arrays no page is looked at)
                src = cache_row(p.block_table, p.max_blocks, p.num_blocks, b, pos);
                dst = cache_row(p.new_table, p.new_max_blocks, p.new_num_blocks, b, j);
            }
            bad = p.n_arrays > 0 && (src < 0 || dst < 0);
            if (p.new_weight) p.new_weight[(int64_t)b * p.new_stride + j] = __ldg(p.weight + (int64_t)b * p.stride + pos);
        }
        if (bad) {
            src = -1;
            atomicCAS(p.status, 0u, (uint32_t)kStBounds);
        }
        s_src[threadIdx.x] = src;
        s_dst[threadIdx.x] = dst;
    }
    __syncthreads();
    for (int k = 0; k < p.n_arrays; ++k) {
        const EvictArray& a = p.arrays[k];
        switch (a.width) {
            case 16: evict_copy_rows<uint4>(a, s_src, s_dst, rows); break;
            case 8: evict_copy_rows<uint2>(a, s_src, s_dst, rows); break;
            case 4: evict_copy_rows<uint32_t>(a, s_src, s_dst, rows); break;
            case 2: evict_copy_rows<uint16_t>(a, s_src, s_dst, rows); break;
            default: evict_copy_rows<uint8_t>(a, s_src, s_dst, rows); break;
        }
    }
}

}  // namespace dsa
