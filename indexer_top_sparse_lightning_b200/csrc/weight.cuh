// weight.cuh -- the attention weight that each cached position draws from new
// tokens (sm_100a):
//
//   w[b, s] = decay * w[b, s] + sum over new tokens t of b and heads h
//             of exp(scale * q[t,h] . row_s[0:576] - lse[t,h])   (s <= t's position)
//
// with lse the log-sum-exp that the attention returned: the sum of the softmax
// weights at s, without the value product.
//
// Per tile of NR (token, head) rows and block of 256 positions a pair of CTAs runs
// one two-CTA product with the POSITIONS on the MMA's M side (128 per CTA: A) and
// the rows on its N side (NR / 2 per CTA's B): a thread then owns a position, and
// its sum over the rows needs no exchange between lanes.  Q stays in shared
// memory for a run of blocks, keys stream through a ring, and the exponentials of
// one block (two warps per lane quarter, half of the rows each) run under the
// MMAs of the next through two score buffers.
//
// NR is 128 when every sequence's new tokens fit one tile (a decode step of 128
// heads): the sums are then complete and are added to w in place.  Otherwise NR
// is 256, which halves the key traffic per product, and each (tile, position) sum
// goes to a scratch row of the tile; weight_sum_kernel adds the rows in tile
// order, so that the result does not depend on which CTA was first.
//
// What bounds it: a decode step reads every latent row once (HBM); chunks are bound
// by the MMAs, 2 * 576 * NR operations per position and tile, with one exponential
// per (row, position) under them.  32 tokens over 32K positions each take 227 to 240 us, 5.2 TB/s of
// the 6.56 of a plain copy; chunks of 150 to 300 tokens of 64 heads over 5K to 9K positions
// 268 to 272 us, 1.13 PFLOP/s.  Over an FP8 cache both read an fp16 copy of the rows that the call makes
// first (596 bytes a position read, 2304 written and read again, and twice the MMAs for the two
// values of an element): 1190 and 580 us.
//
// Roles per CTA (352 threads): warps 0-7 exponentials and sums (lane L of the
// quarter <-> position 128c + L of the block); warp 8 TMEM allocation, in CTA 0 the
// MMA issuer; warp 9 key loads; warp 10 runs and the loads of Q.
#pragma once
#include "common.h"
#include "pair.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

namespace dsa {

template <int NR>
struct WeightCfg {
    static constexpr int BLOCK = 256;                    // positions of a block (two pages per CTA)
    static constexpr int GROUP = NR == 128 ? 3 : 1;      // 64-column chunks of keys that are announced together
    static constexpr int RING = NR == 128 ? 3 : 4;       // such groups that are kept
    static constexpr int CHUNK = 128 * 128;              // 128 positions x 64 columns
    static constexpr int Q_CHUNK = NR / 2 * 128;         // this CTA's rows x 64 columns
    static constexpr int Q_BYTES = 9 * Q_CHUNK;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + Q_BYTES;
    static constexpr int OFF_LSE = OFF_K + RING * GROUP * CHUNK;   // two runs' (factor, -lse) per row
    static constexpr int OFF_SUM = OFF_LSE + 2 * NR * 8;           // two blocks' sums of the second warp of a quarter
    static constexpr int OFF_MISC = OFF_SUM + 2 * 128 * 4;
    static constexpr int MISC_BYTES = 1024;
    static constexpr int SMEM = 1024 + OFF_MISC + MISC_BYTES;
    static constexpr int SUM_WARPS = 8;
    static constexpr int MMA_WARP = 8, KEY_WARP = 9, RUN_WARP = 10;
    static constexpr int THREADS = 352;
    static constexpr int NSEG = 4;
    static constexpr int TMEM_COLS = 2 * NR;
    static constexpr uint32_t idesc(bool f16) {
        return idesc_bf16_f32(256, NR, false, false) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
    }
    using Tiles = TileList<NR, BLOCK>;
};
static_assert(WeightCfg<128>::SMEM <= 232448 && WeightCfg<256>::SMEM <= 232448, "shared memory exceeds the per-CTA limit");

struct WeightParams : ListParams {
    const float* lse;         // [T, H]
    const float* q_factor;    // fp16 queries: the power-of-two factor of each (token, head) row
    const float* page_scale;  // fp16 copy: that of each page
    float* weight;            // [B, stride]
    float* part;              // null: add to `weight`; else [B, tiles_per_seq, part_stride] sums per tile
    int64_t stride, part_stride;
    uint32_t* status;
    int32_t tiles_per_seq;
    float scale_log2, decay;
};

struct WeightMisc {
    uint64_t k_full[4], k_empty[4];      // (full: CTA 0, both CTAs' bytes)
    uint64_t q_full, q_empty;
    uint64_t s_full[2], s_empty[2];
    uint64_t drain;
    uint64_t seg_full[4], seg_empty[4];
    TileRun seg[4];
    uint64_t wait_ns;
    ShareStart start;
    int64_t sums[WeightCfg<128>::THREADS / 32];
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(WeightMisc) <= WeightCfg<128>::MISC_BYTES, "misc block exceeds its slot");

template <int NR, bool F16>
__global__ void __launch_bounds__(WeightCfg<NR>::THREADS, 1)
    attn_weight_kernel(const __grid_constant__ WeightParams p, const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k) {
    using Cfg = WeightCfg<NR>;
    using Tiles = typename Cfg::Tiles;
    constexpr int CHUNKS = F16 ? 18 : 9;                 // of a key row (the fp16 copy: values, then the rest)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_shared(smem_raw, 1024);
    uint8_t* s_q = smem + Cfg::OFF_Q;
    uint8_t* s_k = smem + Cfg::OFF_K;
    float2* s_row = reinterpret_cast<float2*>(smem + Cfg::OFF_LSE);
    float* s_sum = reinterpret_cast<float*>(smem + Cfg::OFF_SUM);
    WeightMisc* m = reinterpret_cast<WeightMisc*>(smem + Cfg::OFF_MISC);
    volatile int* abort = &m->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    int np = (int)(gridDim.x >> 1);
    const int pair = (int)(blockIdx.x >> 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::RING; ++i) {
            mbar_init(&m->k_full[i], 1);
            mbar_init(&m->k_empty[i], 1);
        }
        mbar_init(&m->q_full, 2);
        mbar_init(&m->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->s_empty[i], 2 * Cfg::SUM_WARPS);
        }
        mbar_init(&m->drain, 1);
        for (int i = 0; i < Cfg::NSEG; ++i) {
            mbar_init(&m->seg_full[i], 1);
            mbar_init(&m->seg_empty[i], Cfg::SUM_WARPS + (crank == 0 ? 2 : 1));
        }
        m->abort = 0;
        m->start.b = -1;
        fence_mbar_init();
    }
    if (warp == Cfg::MMA_WARP) {
        tmem_alloc_2cta(&m->tmem_base, Cfg::TMEM_COLS);
        tmem_relinquish_2cta();
    }
    if (warp == Cfg::RUN_WARP && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
    }
    griddep_launch_dependents();
    griddep_wait();
    if (threadIdx.x == 0) {
        const uint32_t us = __ldcg(p.status + 1);        // test hook: wait limit in microseconds
        m->wait_ns = us ? (uint64_t)us * 1000u : kWaitTimeoutNs;
    }
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised before any remote arrive
    tc_fence_after();
    const uint32_t tm_s = m->tmem_base;                  // two score buffers of NR columns
    const uint64_t wlim = m->wait_ns;

    int64_t g0, g1, total;
    Tiles::template share<Cfg::THREADS>(p, pair, np, m->sums, &m->start, p.status, g0, g1, total);

    if (warp == Cfg::RUN_WARP) {
        // ---------------------------------------------------------------- runs, loads of Q
        typename Tiles::Walk w = Tiles::begin(p, m->start, g0, g1);
        bool ok = true;
        if (lane == 0) {
            const uint32_t q_full = mapa_shared(smem_u32(&m->q_full), 0);
            for (int ns = 0;; ++ns) {
                const int r = ns % Cfg::NSEG;
                if (!mbar_spin(&m->seg_empty[r], ((ns / Cfg::NSEG) & 1) ^ 1, abort, wlim)) {
                    ok = false;
                    break;
                }
                if (w.g >= w.g1) {
                    m->seg[r].b = -1;
                    mbar_arrive(&m->seg_full[r]);
                    break;
                }
                int64_t nb;
                const TileRun sg = Tiles::run(p, w, nb);
                m->seg[r] = sg;
                mbar_arrive(&m->seg_full[r]);
                // Q, once every product of the run before has completed
                if (ns > 0 && !mbar_spin(&m->q_empty, (ns - 1) & 1, abort, wlim)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx_cluster(q_full, Cfg::Q_BYTES);
                tma_load_3d_pair(s_q, &tm_q, q_full, 0, sg.row0 + NR / 2 * (int)crank, 0);
                Tiles::next(p, w, sg);
            }
            if (!ok) *abort = 1;
        }
        __syncwarp();
    } else if (warp == Cfg::KEY_WARP) {
        // ---------------------------------------------------------------- loads of keys
        const bool el = elect_one();
        bool ok = true, bad = false;
        uint32_t r = 0, ph = 1;
        const uint32_t lead = mapa_shared(smem_u32(&m->k_full[0]), 0);
        TileRun sg = {};
        auto page_id = [&](int page) -> int {            // -1: nobody sees the page; -2: a bad id
            if (page >= p.max_blocks || page * kPage >= sg.see) return -1;
            const int id = __ldg(p.block_table + (int64_t)sg.b * p.max_blocks + page);
            return id >= 0 && id < p.num_blocks ? (p.staged ? sg.b * p.staged + page : id) : -2;
        };
        for (int ns = 0; ok; ++ns) {
            const int sr = ns % Cfg::NSEG;
            if (!elected_wait(el, &m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim)) {
                ok = false;
                break;
            }
            sg = m->seg[sr];
            __syncwarp();
            if (el) mbar_arrive(&m->seg_empty[sr]);
            if (sg.b < 0) break;
            const int k0 = __shfl_sync(0xffffffffu, sg.k0, 0), k1 = __shfl_sync(0xffffffffu, sg.k1, 0);
            // ids of the block's four pages one block ahead: this CTA's are 2 crank, 2 crank + 1
            int id[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) id[i] = page_id(4 * k0 + i);
            for (int k = k0; ok && k < k1; ++k) {
                int next[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) next[i] = page_id(4 * (k + 1) + i);
                int pages = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    bad = bad || id[i] == -2;
                    pages += id[i] >= 0;
                }
                const int i0 = crank == 0 ? id[0] : id[2], i1 = crank == 0 ? id[1] : id[3];
#pragma unroll 1
                for (int c = 0; c < CHUNKS; c += Cfg::GROUP) {
                    if (!elected_wait(el, &m->k_empty[r], ph, abort, wlim)) {
                        ok = false;
                        break;
                    }
                    // a page that nobody sees is not loaded: its positions' sums are not used
                    if (crank == 0 && el) mbar_arrive_expect_tx(&m->k_full[r], pages * Cfg::GROUP * (Cfg::CHUNK / 2));
                    uint8_t* dst = s_k + r * (Cfg::GROUP * Cfg::CHUNK);
                    // (fp16: the small rests first, so that adding them up costs no bits of the sum)
                    const int z = F16 ? (c < 9 ? c + 9 : c - 9) : c;
#pragma unroll
                    for (int j = 0; j < Cfg::GROUP; ++j) {
                        if (el && i0 >= 0) tma_load_3d_pair(dst + j * Cfg::CHUNK, &tm_k, lead + 8 * r, 0, i0 * kPage, z + j);
                        if (el && i1 >= 0)
                            tma_load_3d_pair(dst + j * Cfg::CHUNK + Cfg::CHUNK / 2, &tm_k, lead + 8 * r, 0, i1 * kPage, z + j);
                    }
                    if (++r == Cfg::RING) {
                        r = 0;
                        ph ^= 1;
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) id[i] = next[i];
            }
        }
        if (bad && el) atomicCAS(p.status, 0u, (uint32_t)kStBounds);
        if (!ok) *abort = 1;
    } else if (warp == Cfg::MMA_WARP) {
        if (crank == 0) {
            // ------------------------------------------------------------ MMA issuer
            const bool el = elect_one();
            bool ok = true;
            const uint64_t q_desc = sdesc_sw128(smem_u32(s_q), 16, 1024);
            const uint64_t k_desc = sdesc_sw128(smem_u32(s_k), 16, 1024);
            uint32_t blk = 0, r = 0, ph = 0;
            for (int ns = 0; ok; ++ns) {
                const int sr = ns % Cfg::NSEG;
                if (!elected_wait(el, &m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim)) {
                    ok = false;
                    break;
                }
                const TileRun sg = m->seg[sr];
                __syncwarp();
                if (el) mbar_arrive(&m->seg_empty[sr]);
                if (sg.b < 0) break;
                ok = elected_wait(el, &m->q_full, ns & 1, abort, wlim);
                const int nb = __shfl_sync(0xffffffffu, sg.k1 - sg.k0, 0);
                for (int i = 0; ok && i < nb; ++i, ++blk) {
                    ok = elected_wait(el, &m->s_empty[blk & 1], ((blk >> 1) & 1) ^ 1, abort, wlim);
                    tc_fence_after();
                    const uint32_t d = tm_s + (blk & 1) * NR;
                    uint32_t q_off = 0;
#pragma unroll 1
                    for (int c = 0; ok && c < CHUNKS; c += Cfg::GROUP) {
                        ok = elected_wait(el, &m->k_full[r], ph, abort, wlim);
                        if (!ok) break;
                        const uint64_t kd = k_desc + r * (Cfg::GROUP * Cfg::CHUNK / 16);
#pragma unroll
                        for (int j = 0; j < 4 * Cfg::GROUP; ++j)
                            if (el)
                                umma_bf16_2cta(d, kd + ((j >> 2) * (Cfg::CHUNK / 16) + (j & 3) * 2),
                                               q_desc + q_off + ((j >> 2) * (Cfg::Q_CHUNK / 16) + (j & 3) * 2), Cfg::idesc(F16),
                                               (c | j) != 0);
                        if (el) umma_commit_2cta(&m->k_empty[r], 3);
                        if (++r == Cfg::RING) {
                            r = 0;
                            ph ^= 1;
                        }
                        // the copy's second half meets the same columns of Q
                        q_off = c + Cfg::GROUP == 9 ? 0 : q_off + Cfg::GROUP * (Cfg::Q_CHUNK / 16);
                    }
                    if (el) umma_commit_2cta(&m->s_full[blk & 1], 3);
                    if (i + 1 == nb && el) umma_commit_2cta(&m->q_empty, 3);
                }
            }
            volatile int no_abort = 0;
            if (el) {
                umma_commit_2cta(&m->drain, 1);
                mbar_spin(&m->drain, 0, &no_abort, wlim);
            }
            __syncwarp();
            if (!ok) *abort = 1;
        }
    } else {
        // ---------------------------------------------------------------- exponentials and sums
        const int L = threadIdx.x & 127;                 // position of this CTA's 128 of a block
        const int part = threadIdx.x >> 7;               // rows NR/2 * part ..
        constexpr int COLS = NR / 2;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        uint32_t blk = 0;
        bool ok = true;
        // Every exit decision of these 256 threads is taken together (votes carried by named
        // barriers), so the named barriers always match.
        for (int ns = 0;; ++ns) {
            const int sr = ns % Cfg::NSEG;
            const bool there = warp_wait(&m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim);
            ok = named_bar_and(1, 256, ok && there);
            if (!ok) break;
            const TileRun sg = m->seg[sr];
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->seg_empty[sr]);
            if (sg.b < 0) break;
            // the rows' log-sum-exps in log2 units; a row that saw nothing (-inf) adds nothing
            float2* row = s_row + (ns & 1) * NR;
            bool dead = false;
            if ((int)threadIdx.x < NR) {
                float2 v = make_float2(0.0f, -INFINITY);
                if ((int)threadIdx.x < sg.nrows) {
                    const float l = __ldg(p.lse + (int64_t)sg.row0 + threadIdx.x);
                    v.x = p.scale_log2;
                    if constexpr (F16) v.x *= __ldg(p.q_factor + (int64_t)sg.row0 + threadIdx.x);
                    dead = l == -INFINITY;
                    v.y = dead ? -INFINITY : -l * 1.4426950408889634f;
                }
                row[threadIdx.x] = v;
            }
            const bool alive = named_bar_and(1, 256, !dead);     // (of the tile's real rows)
            for (int k = sg.k0; k < sg.k1; ++k, ++blk) {
                const uint32_t b = blk & 1;
                const int pos = k * Cfg::BLOCK + 128 * (int)crank + L;
                // rows that see the position: those of tokens at or behind it
                const int64_t behind = (int64_t)(pos - sg.c) * p.H - ((int64_t)sg.tok * p.H + sg.head);
                const int first = behind < 0 ? 0 : behind > NR ? NR : (int)behind;
                const int page = pos / kPage;
                bool there_is = pos < sg.see && page < p.max_blocks;
                float f = 1.0f;
                if (there_is) {
                    const int id = __ldg(p.block_table + (int64_t)sg.b * p.max_blocks + page);
                    there_is = id >= 0 && id < p.num_blocks;
                    if constexpr (F16) f = __ldg(p.page_scale + (int64_t)sg.b * p.staged + page);
                }
                bool got = ok && warp_wait(&m->s_full[b], (blk >> 1) & 1, abort, wlim);
                float sum = 0.0f;
                if (got) {
                    tc_fence_after();
                    const bool all = __all_sync(0xffffffffu, first == 0) && sg.nrows == NR && alive;
                    float a0 = 0.0f, a1 = 0.0f, a2 = 0.0f, a3 = 0.0f;
#pragma unroll 1
                    for (int c0 = COLS * part; c0 < COLS * (part + 1); c0 += 32) {
                        uint32_t x[32];
                        tmem_ld32(tm_s + lane_off + b * NR + c0, x);
                        tmem_wait_ld();
                        const float4* rw = reinterpret_cast<const float4*>(row + c0);   // two rows each
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 u = rw[i / 2], v = rw[i / 2 + 1];
                            float e[4];
                            e[0] = fast_exp2(fmaf(__uint_as_float(x[i]), u.x * f, u.y));
                            e[1] = fast_exp2(fmaf(__uint_as_float(x[i + 1]), u.z * f, u.w));
                            e[2] = fast_exp2(fmaf(__uint_as_float(x[i + 2]), v.x * f, v.y));
                            e[3] = fast_exp2(fmaf(__uint_as_float(x[i + 3]), v.z * f, v.w));
                            if (!all) {
                                // rows of other sequences, rows in front of the position and rows that saw
                                // nothing: whatever the scores are there, they are not added
                                const float off[4] = {u.y, u.w, v.y, v.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    if (c0 + i + j < first || off[j] == -INFINITY) e[j] = 0.0f;
                            }
                            a0 += e[0];
                            a1 += e[1];
                            a2 += e[2];
                            a3 += e[3];
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader(&m->s_empty[b], crank);
                    sum = (a0 + a1) + (a2 + a3);
                }
                if (part == 1) s_sum[b * 128 + L] = sum;
                ok = named_bar_and(1, 256, got);
                if (!ok) break;
                if (part == 0) {
                    sum += s_sum[b * 128 + L];
                    if (!there_is) sum = 0.0f;
                    if (p.part) {
                        if (pos < p.part_stride)
                            p.part[((int64_t)sg.b * p.tiles_per_seq + sg.tile) * p.part_stride + pos] = sum;
                    } else if (pos < sg.see) {
                        float* w = p.weight + (int64_t)sg.b * p.stride + pos;
                        *w = p.decay == 0.0f ? sum : fmaf(p.decay, *w, sum);
                    }
                }
            }
            if (!ok) break;
        }
        if (!ok) *abort = 1;
    }

    // ---------------------------------------------------------------- teardown
    tc_fence_before();
    __syncthreads();
    // given up: copies still in flight land within microseconds; wait far longer than that
    if (m->abort)
        for (int i = 0; i < 100; ++i) __nanosleep(10000);
    cluster_sync();   // no remote access may target an exited CTA, and no MMA may read a freed tile
    if (warp == Cfg::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_2cta(m->tmem_base, Cfg::TMEM_COLS);
    }
    if (threadIdx.x == 0 && m->abort) atomicCAS(p.status, 0u, (uint32_t)kStTimeout);
}

// w = decay * w + the tiles' sums, in tile order: one thread per position.  Tile i of
// a sequence covers a position when its blocks reach it; the tiles are in the order
// of their tokens, so those that do are the last ones.
constexpr int kWeightSumThreads = 256;

template <int NR>
__global__ void __launch_bounds__(kWeightSumThreads) weight_sum_kernel(const __grid_constant__ WeightParams p) {
    using Tiles = typename WeightCfg<NR>::Tiles;
    griddep_wait();
    const int b = (int)blockIdx.y;
    const int pos = (int)blockIdx.x * kWeightSumThreads + (int)threadIdx.x;
    bool ok;
    const ChunkSeq s = Tiles::seq(p, b, ok);
    if (s.tiles == 0 || pos >= s.len) return;            // no new tokens (in this window): unchanged
    // blocks(i) = (i + 1 + first) / (G H) + 1 > pos / BLOCK for i < tiles - 1
    const int64_t need = (int64_t)(pos / WeightCfg<NR>::BLOCK) * Tiles::G * p.H - 1 - s.first;
    int i = need <= 0 ? 0 : need < s.tiles - 1 ? (int)need : s.tiles - 1;
    if (pos >= (int64_t)Tiles::blocks(s, p.H, s.tiles - 1) * WeightCfg<NR>::BLOCK) i = s.tiles;   // nobody sees it yet
    const float* src = p.part + (int64_t)b * p.tiles_per_seq * p.part_stride + pos;
    float sum = 0.0f;
    for (; i + 4 <= s.tiles; i += 4) {
        const float x0 = __ldcg(src + (int64_t)i * p.part_stride), x1 = __ldcg(src + (int64_t)(i + 1) * p.part_stride);
        const float x2 = __ldcg(src + (int64_t)(i + 2) * p.part_stride), x3 = __ldcg(src + (int64_t)(i + 3) * p.part_stride);
        sum = (((sum + x0) + x1) + x2) + x3;
    }
    for (; i < s.tiles; ++i) sum += __ldcg(src + (int64_t)i * p.part_stride);
    float* w = p.weight + (int64_t)b * p.stride + pos;
    *w = p.decay == 0.0f ? sum : fmaf(p.decay, *w, sum);
}

}  // namespace dsa
