// chunk.cuh -- dense attention of new tokens over the paged MLA latent cache
// (sm_100a): every new token attends to all positions up to its own.
//
// For new token j of a sequence with cached length L and n new tokens, at
// position p = L - n + j, and each of its H heads:
//   S_s = scale * q . row_s[0:576]  (s = 0..p),  P = softmax(S),
//   O = sum_s P_s row_s[0:512],  lse = log sum_s exp(S_s).
//
// Tiles and blocks.  The (token, head) rows of a sequence, token-major, are cut
// into tiles of 128 rows (one token of 128 heads, eight of 16, ...), and the
// positions a tile sees into blocks of 128 (two pages).  All blocks of all
// tiles form one list; each cluster of two CTAs ("pair") takes an even,
// contiguous share of it, so that the SMs finish together whatever the lengths.
// A tile whose blocks are spread over several pairs leaves one partial result
// per pair (unnormalized O, running maximum and sums, all fp32), merged by
// chunk_combine_kernel.
//
// Per block the pair runs two-CTA tensor-core MMAs (tcgen05 cta_group::2,
// issued by CTA 0):
//   S = Q.K^T: M = 128 rows (64 per CTA), N = 128 positions (CTA c holds page
//       2k + c), nine K-chunks of 64 columns;
//   O += P.V: M = 128 rows, N = 256 value columns twice (CTA c holds columns
//       256c.. of both pages; MMA h takes 128 of them from each CTA, columns
//       128h.. and 256 + 128h..), K = 128 positions.
// Keys and values have a ring each (a block of keys in three groups of 64 rows x
// 192 columns; of values, three groups of 32 rows x 256 of the pair's 512 columns,
// four make a block), a loading warp each and an issuing warp each: one
// warp cannot issue a block's 52 MMAs and wait for their operands in the time
// that the MMAs take.  The issuing warps run ahead of one another as far as the
// two score buffers and the two weight buffers allow, across tiles too, so the
// softmax of one block runs under the products of its neighbours.  Every group is
// one or two copies (the tensor maps have the 64-column chunks of a row as their
// outermost dimension), counted for both CTAs on CTA 0's barriers (the two-CTA
// form of the tiled load), which CTA 0's loaders arm for both.
//
// What bounds it.  2176 * 128 * 128 operations per block of the pair take about
// 1.15 us at the tensor core's rate, and the block's operands are 278 KB through
// L2 (each CTA needs its page whole, and its half of the value columns of both):
// at chunk lengths the L2 path and the MMAs are about even, and a decode step
// of 128 heads sits at the ridge of HBM and tensor rate.  The last 2048 tokens of a
// 16K prompt take 7.15 to 7.35 ms, 1.19 to 1.22 PFLOP/s (cuBLAS holds 1.38 for as long; the clock is
// at the power limit); 32 tokens over 32K positions each 340 to 370 us, 3.3 to 3.6 TB/s and 0.79
// to 0.86 PFLOP/s at once (at 1.30 GHz when the calls go on for seconds; the merge ends 21 us after
// the attention), of 16 heads 290; one token at 4K 16.6 us, most of it start, planning and merge.
//
// Masked positions.  Scores past a row's own position are replaced, not
// multiplied.  In P.V a weight of zero still multiplies the value row, so rows
// that nobody in the tile sees (the tail of the last page, which may hold
// anything, NaN included) are overwritten with zeros in shared memory, and
// non-finite rows that only some of the tile's tokens see are zeroed too (the
// tokens that see one have a non-finite score already).  Only the slots at the
// tile's causal edge take this path (the "fixer" warp).
//
// Roles per CTA (448 threads; over an FP8 cache 768):
//   warps 0-7   softmax and epilogue (warps w and w + 4 share TMEM lanes 32(w%4)..;
//               lane L: row 64c + L%64, positions 64*(L/64).. of a block)
//   warp 8      TMEM allocation; CTA 0: issues the score MMAs
//   warp 9      CTA 0: issues the value MMAs
//   warps 10, 11  loads of keys, of values
//   warp 12     segments (runs of one tile's blocks) and the loads of Q
//   warp 13     fixer
// Over an FP8 cache (chunk_fp8.cuh): warp 10 segments and Q, 11 and 12 loads of the codes of
// keys, of values, 13 and 14 position factors, 16-19 conversion of keys, 20-23 of values.
#pragma once
#include "chunk_cfg.cuh"
#include "chunk_fp8.cuh"

namespace dsa {

// An FP8 cache (e4m3 codes) meets fp16 operands, and Q is brought to fp16 in shared memory:
// both operands of an MMA have one type, and bf16 would round the products of codes and
// scales eight times as far.  A power of two per row of Q keeps it in fp16's range.  The
// operands are made by chunk_fp8.cuh, which leaves four score accumulators to be put together
// here, or read from the fp16 copy of latent.cu (many tiles over few positions: the copy stays
// in L2, and a code is converted once), whose rows hold the rounded values and what their
// rounding left out: the scores take both, with twice the score MMAs and key loads.  With
// t_s = S_s + log2 F_s (F_s the page's power of two) the weights that multiply the values
// code * f / F are P_s F_s = 2^(t_s - m), so the reference m follows t, and the sums of
// weights are those of 2^(t_s - m) / F_s.
template <ChunkCache CACHE>
__global__ void __launch_bounds__(32 * ChunkCfg::warps(CACHE == kCacheFp8), 1)
    chunk_attn_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ CUtensorMap tm_r) {
    using Cfg = ChunkCfg;
    constexpr bool FP8 = CACHE == kCacheFp8, COPY = CACHE == kCacheCopy, F16 = CACHE != kCacheBf16;
    constexpr int SMW = Cfg::SOFTMAX_WARPS, QK_WARP = SMW, PV_WARP = SMW + 1;
    constexpr int KEY_WARP = SMW + 2, VALUE_WARP = SMW + 3, FIX_WARP = SMW + 5;
    constexpr int KLOAD_WARP = SMW + 3, FACTOR_WARP = SMW + 5;   // FP8: two loading warps, two of factors
    constexpr int FKEY_WARP = SMW + 8, FVALUE_WARP = FKEY_WARP + Cfg::CONV_WARPS;
    constexpr int SEG_WARP = FP8 ? SMW + 2 : SMW + 4;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_shared(smem_raw, 1024);
    uint8_t* s_q = smem + Cfg::OFF_Q;
    uint8_t* s_p = smem + Cfg::OFF_P;
    uint8_t* s_k = smem + (FP8 ? Cfg::OFF_FK : Cfg::OFF_K);
    uint8_t* s_v = smem + (FP8 ? Cfg::OFF_FV : Cfg::OFF_V);
    ChunkScales* s_rec = reinterpret_cast<ChunkScales*>(smem + Cfg::OFF_REC);
    float* s_xm = reinterpret_cast<float*>(smem + (FP8 ? kChunkFp8Xm : Cfg::OFF_XM));
    ChunkMisc* m = reinterpret_cast<ChunkMisc*>(smem + Cfg::OFF_MISC);
    volatile int* abort = &m->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    int np = (int)(gridDim.x >> 1);
    const int pair = (int)(blockIdx.x >> 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::KRING; ++i) {
            mbar_init(&m->k_full[i], FP8 ? 2 : 1);    // CTA 0's loader, for both CTAs; FP8: both CTAs' converters
            mbar_init(&m->k_empty[i], FP8 ? 2 : 1);
        }
        for (int i = 0; i < Cfg::VRING; ++i) {
            mbar_init(&m->v_full[i], FP8 ? 2 : 1);    // ... or fixer
            mbar_init(&m->v_peer[i], 1);
            mbar_init(&m->v_empty[i], FP8 ? 2 : 1);
            mbar_init(&m->v_land[i], 1);
        }
        mbar_init(&m->q_full, F16 ? 2 * SMW : 2);
        mbar_init(&m->q_land, 1);
        mbar_init(&m->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->s_empty[i], 2 * SMW);   // those of both CTAs
            mbar_init(&m->p_full[i], 2 * SMW);
            mbar_init(&m->p_empty[i], 1);
            mbar_init(&m->drain[i], 1);
        }
        mbar_init(&m->o_full, 1);
        mbar_init(&m->o_empty, 2 * SMW);
        for (int i = 0; i < Cfg::NSEG; ++i) {
            mbar_init(&m->seg_full[i], 1);
            // FP8: factors and converting warps; else loading and fixer warps; CTA 0: the issuers too
            mbar_init(&m->seg_empty[i], SMW + (FP8 ? 4 + 2 * Cfg::CONV_WARPS : 3) + (crank == 0 ? 2 : 0));
        }
        for (int i = 0; i < Cfg::NREC; ++i) {
            mbar_init(&m->rec_full[i], 2);
            mbar_init(&m->rec_empty[i], SMW + 2);
        }
        if (FP8) {
            // the operand rings are empty: no MMAs to wait for in their first round
            for (int i = 0; i < Cfg::FKRING; ++i) {
                mbar_init(&m->kc_empty[i], 1);
                mbar_arrive(&m->k_empty[i]);
            }
            for (int i = 0; i < Cfg::FVRING; ++i) {
                mbar_init(&m->vc_empty[i], 1);
                mbar_arrive(&m->v_empty[i]);
            }
        }
        m->abort = 0;
        m->start.b = -1;
        fence_mbar_init();
    }
    if (warp == QK_WARP) {
        tmem_alloc_2cta(&m->tmem_base, Cfg::TMEM_COLS);
        tmem_relinquish_2cta();
    }
    if (warp == SEG_WARP && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        if (FP8) prefetch_tmap(&tm_r);
    }
    // the merge kernel (a programmatic dependent) may be scheduled on SMs this grid
    // leaves idle; it waits for the whole grid before reading anything
    griddep_launch_dependents();
    griddep_wait();
    if (threadIdx.x == 0) {
        // test hooks in the status area: word 1 = wait limit in microseconds (0: the
        // default), word 2 = fault injection bits
        const uint32_t us = __ldcg(p.status + 1);
        m->wait_ns = us ? (uint64_t)us * 1000u : kWaitTimeoutNs;
        m->inject = __ldcg(p.status + 2);
    }
    tc_fence_before();
    cluster_sync();   // barriers of both CTAs initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = m->tmem_base;
    const uint32_t tm_o = tmem_base;            // columns [0, 256)
    const uint32_t tm_s = tmem_base + 256;      // score buffers, 64 columns each (FP8: one, of four times that)
    const uint64_t wlim = m->wait_ns;

    // ---------------------------------------------------------------- this pair's share of the list
    int64_t g0, g1, total;
    ChunkTiles::share<32 * Cfg::warps(FP8)>(p, pair, np, m->sums, &m->start, p.status, g0, g1, total);

    if (warp == SEG_WARP) {
        // ---------------------------------------------------------------- segments, loads of Q
        ChunkTiles::Walk w = ChunkTiles::begin(p, m->start, g0, g1);
        // for the merge: first row, rows and pairs of the tile that starts here and ends in a later pair
        int4 head = make_int4(0, 0, 0, 0);
        bool ok = true;
        int ns = 0;
        if (lane == 0) {
            const uint32_t q_full = mapa_shared(smem_u32(&m->q_full), 0);
            while (true) {
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
                const TileRun sg = ChunkTiles::run(p, w, nb);
                m->seg[r] = sg;
                mbar_arrive(&m->seg_full[r]);
                if (sg.part == 1)
                    head = make_int4(sg.row0, sg.nrows, share_of(total, w.tile_g0 + nb - 1, np) - pair + 1, 0);
                // Q, once every QK of the segment before has completed
                if (ns > 0 && !mbar_spin(&m->q_empty, (ns - 1) & 1, abort, wlim)) {
                    ok = false;
                    break;
                }
                if constexpr (F16) {
                    mbar_arrive_expect_tx(&m->q_land, Cfg::Q_BYTES);
                    tma_load_3d(s_q, &tm_q, &m->q_land, 0, sg.row0 + 64 * (int)crank, 0);
                } else {
                    mbar_arrive_expect_tx_cluster(q_full, Cfg::Q_BYTES);
                    tma_load_3d_pair(s_q, &tm_q, q_full, 0, sg.row0 + 64 * (int)crank, 0);
                }
                ++ns;
                ChunkTiles::next(p, w, sg);
            }
            if (!ok) *abort = 1;
            if (crank == 0) reinterpret_cast<int4*>(p.part)[pair] = head;
        }
        __syncwarp();
    } else if (FP8 && warp >= KLOAD_WARP) {
        // ---------------------------------------------------------------- an FP8 cache: codes, factors, keys, values
        const int ti = (int)threadIdx.x - 32 * (warp < FVALUE_WARP ? FKEY_WARP : FVALUE_WARP);
        bool ok = !(crank == 1 && (m->inject & 4u));   // test hook: the second CTA never loads
        if (ok && warp != FACTOR_WARP + 2)
            ok = warp < FACTOR_WARP   ? fp8_codes(p, m, smem, tm_k, tm_r, tm_v, warp == KLOAD_WARP, crank, abort, wlim)
                 : warp < FKEY_WARP   ? fp8_factors(p, m, s_rec, warp - FACTOR_WARP, crank, abort, wlim)
                 : warp < FVALUE_WARP ? fp8_keys(p, m, smem, ti, crank, abort, wlim)
                                      : fp8_values(p, m, smem, ti, crank, abort, wlim);
        if (!ok) *abort = 1;
    } else if (!FP8 && (warp == KEY_WARP || warp == VALUE_WARP)) {
        // ---------------------------------------------------------------- loads of keys, of values
        // The whole warp runs the schedule and one elected lane acts, so that addresses and
        // coordinates stay in uniform registers (per-lane values would have to be moved there for
        // every copy).  CTA 0 announces the bytes of both CTAs (both see the same page ids), so
        // that CTA 1 only issues its copies.
        const bool keys = warp == KEY_WARP;
        const bool el = elect_one();
        // test hook: the second CTA never loads
        bool ok = !(crank == 1 && (m->inject & 4u));
        bool bad = false;
        uint32_t r = 0, ph = 1;            // group of the (value) ring and the parity that its `empty` waits for
        const uint32_t k_lead = mapa_shared(smem_u32(&m->k_full[0]), 0), v_lead = mapa_shared(smem_u32(&m->v_full[0]), 0);
        TileRun sg = {};
        const int32_t* table = nullptr;
        auto page_id = [&](int page) -> int {
            const int id = chunk_page(p, sg, table, page);
            return COPY && id >= 0 ? sg.b * p.staged + page : id;
        };
        auto load_keys = [&](int id0, int id1) -> bool {
            const int id = crank == 0 ? id0 : id1;
            // a page that nobody sees is not loaded: its scores are replaced whatever they are
            const uint32_t bytes = (uint32_t)Cfg::KGROUP * ((id0 >= 0) + (id1 >= 0));
            const bool mine = el && id >= 0;
            const int y = id * kPage;
#pragma unroll 1
            for (int g = 0; g < (COPY ? 2 : 1) * Cfg::KRING; ++g) {
                const int kr = g % Cfg::KRING;
                if (!elected_wait(el, &m->k_empty[kr], ph, abort, wlim)) return false;
                if (crank == 0 && el) mbar_arrive_expect_tx(&m->k_full[kr], bytes);
                // (the copy's small rests first, so that adding them up costs no bits of the sum)
                const int chunk = !COPY ? 3 * g : g < Cfg::KRING ? 3 * g + 9 : 3 * g - 9;
                if (mine) tma_load_3d_pair(s_k + kr * Cfg::KGROUP, &tm_k, k_lead + 8 * kr, 0, y, chunk);
                if (kr == Cfg::KRING - 1) ph ^= 1;
            }
            return true;
        };
        auto next_group = [&]() {
            if (++r == Cfg::VRING) {
                r = 0;
                ph ^= 1;
            }
        };
        // Four groups of 32 positions, both pages good, nothing for the fixer.
        auto load_values = [&](int id0, int id1) -> bool {
#pragma unroll 1
            for (int g = 0; g < Cfg::VGROUPS; ++g) {
                if (!elected_wait(el, &m->v_empty[r], ph, abort, wlim)) return false;
                if (crank == 0 && el) mbar_arrive_expect_tx(&m->v_full[r], 2 * Cfg::VGROUP);
                const int y = (g < 2 ? id0 : id1) * kPage + 32 * (g & 1);
                if (el) tma_load_3d_pair(s_v + r * Cfg::VGROUP, &tm_v, v_lead + 8 * r, 0, y, 4 * (int)crank);
                next_group();
            }
            return true;
        };
        // The same at the causal edge (the groups that the fixer looks at first), or with a bad
        // page: all groups of such a block go through the fixer's hands.
        auto load_values_edge = [&](const ChunkBlock& cb, int id0, int id1) -> bool {
#pragma unroll 1
            for (int g = 0; g < cb.ngroups; ++g, next_group()) {
                if (!elected_wait(el, &m->v_empty[r], ph, abort, wlim)) return false;
                const int id = g < 2 ? id0 : id1;
                uint8_t* dst = s_v + r * Cfg::VGROUP;
                if (id < 0) {              // a bad page id: zeros
                    for (int i = lane; i < Cfg::VGROUP / 16; i += 32)
                        reinterpret_cast<uint4*>(dst)[i] = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (!el) continue;
                if (id >= 0) {
                    mbar_arrive_expect_tx(&m->v_land[r], Cfg::VGROUP);
                    tma_load_3d(dst, &tm_v, &m->v_land[r], 0, id * kPage + 32 * (g & 1), 4 * (int)crank);
                } else {
                    mbar_arrive(&m->v_land[r]);
                }
            }
            return true;
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
            table = p.block_table + (int64_t)sg.b * p.max_blocks;
            const int k0 = __shfl_sync(0xffffffffu, sg.k0, 0), k1 = __shfl_sync(0xffffffffu, sg.k1, 0);
            // page ids one block ahead, so that no load waits for one.  (Asking for the pages in L2
            // three blocks ahead made a decode step slower, 362 -> 432 us by lines, 477 by pages.)
            int a0 = page_id(2 * k0), a1 = page_id(2 * k0 + 1);
            for (int k = k0; ok && k < k1; ++k) {
                const int b0 = page_id(2 * k + 2), b1 = page_id(2 * k + 3);
                if (keys) {
                    bad = bad || a0 == -2 || a1 == -2;
                    ok = load_keys(a0, a1);
                } else {
                    const ChunkBlock cb = chunk_block(sg, k);
                    const bool plain = __all_sync(0xffffffffu, cb.fix_from == Cfg::VGROUPS && a0 >= 0 && a1 >= 0);
                    ok = plain ? load_values(a0, a1) : load_values_edge(cb, a0, a1);
                }
                a0 = b0;
                a1 = b1;
            }
        }
        if (bad && el) atomicCAS(p.status, 0u, (uint32_t)kStBounds);
        if (!ok) *abort = 1;
    } else if (!FP8 && warp == FIX_WARP) {
        // ---------------------------------------------------------------- value rows at the causal edge
        bool ok = true;
        uint32_t n = 0, phase = 0, peer = 0;   // groups so far; next phase of each land and peer barrier
        for (int ns = 0; ok; ++ns) {
            const int sr = ns % Cfg::NSEG;
            if (!warp_wait(&m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim)) {
                ok = false;
                break;
            }
            const TileRun sg = m->seg[sr];
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->seg_empty[sr]);
            if (sg.b < 0) break;
            // the loader's rule for the blocks that it hands over: lanes 2i and 2i + 1 look at the
            // pages of block kb + i
            const int32_t* table = p.block_table + (int64_t)sg.b * p.max_blocks;
            int kb = sg.k0 - 16;
            uint32_t good = 0;
            auto pages_ok = [&](int k) -> bool {
                if (k >= kb + 16) {
                    kb = k;
                    const int page = 2 * k + lane;
                    bool fine = true;
                    if (page < p.max_blocks && page * kPage < sg.see) {
                        const int id = __ldg(table + page);
                        fine = id >= 0 && id < p.num_blocks;
                    }
                    good = __ballot_sync(0xffffffffu, fine);
                }
                return ((good >> (2 * (k - kb))) & 3u) == 3u;
            };
            for (int k = sg.k0; ok && k < sg.k1; ++k) {
                const ChunkBlock cb = chunk_block(sg, k);
                if (cb.fix_from == Cfg::VGROUPS && pages_ok(k)) {
                    n += Cfg::VGROUPS;
                    continue;
                }
                for (int g = 0; ok && g < cb.ngroups; ++g, ++n) {
                    const uint32_t r = n % Cfg::VRING;
                    ok = warp_wait(&m->v_land[r], (phase >> r) & 1, abort, wlim);
                    if (!ok) break;
                    phase ^= 1u << r;
                    // lane = row of the group: four 64-column chunks of 128 bytes, 4096 apart, their
                    // 16-byte parts in an order that spreads the lanes over the banks
                    uint8_t* row = s_v + r * Cfg::VGROUP + lane * 128;
                    auto part = [&](int q) -> uint4* {
                        return reinterpret_cast<uint4*>(row + (q >> 3) * 4096 + (((q + lane) & 7) << 4));
                    };
                    const int pos = k * Cfg::BLOCK + 32 * g + lane;
                    bool zero = pos >= sg.see;
                    if (!zero && pos >= sg.see_all) {
                        constexpr uint32_t EXP = F16 ? 0x7C00u : 0x7F80u;
                        uint32_t odd = 0;  // an exponent of all ones
#pragma unroll 1
                        for (int q = 0; q < 32; ++q) {
                            const uint4 v = *part(q);
                            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                odd |= (uint32_t)((w[e] & EXP) == EXP) | (uint32_t)((w[e] & (EXP << 16)) == (EXP << 16));
                        }
                        zero = odd != 0;
                    }
                    if (zero)
#pragma unroll 1
                        for (int q = 0; q < 32; ++q) *part(q) = make_uint4(0u, 0u, 0u, 0u);
                    fence_proxy_async_smem();
                    __syncwarp();
                    // CTA 0's fixer hands the group over once both have looked at it
                    if (crank == 1) {
                        if (lane == 0) mbar_arrive_remote(mapa_shared(smem_u32(&m->v_peer[r]), 0));
                    } else {
                        ok = warp_wait(&m->v_peer[r], (peer >> r) & 1, abort, wlim);
                        peer ^= 1u << r;
                        if (ok && lane == 0) mbar_arrive(&m->v_full[r]);
                    }
                }
            }
        }
        if (!ok) *abort = 1;
    } else if (warp == QK_WARP || warp == PV_WARP) {
        // ---------------------------------------------------------------- MMA issuers (CTA 0)
        // The whole warp runs the schedule and one elected lane issues, so that the operand
        // descriptors stay in uniform registers: 30 cycles per MMA where descriptors kept per
        // lane cost 51 (the MMAs themselves take 32 and 64).  Descriptors differ from a base by
        // multiples of 16 bytes in their low words.
        const bool qk = warp == QK_WARP;
        if (crank == 0) {
            const bool el = elect_one();
            bool ok = true;
            const uint64_t q_desc = sdesc_sw128(smem_u32(s_q), 16, 1024);
            const uint64_t k_desc = sdesc_sw128(smem_u32(s_k), 16, 1024);
            const uint64_t p_desc = sdesc_sw128(smem_u32(s_p), 16, 1024);
            // V [16 positions x 128 columns per CTA] MN-major: 64-column chunks of 32 rows 4096 B
            // apart (LBO), 8-row groups 1024 B (SBO)
            const uint64_t v_desc = sdesc_sw128(smem_u32(s_v), 4096, 1024);
            uint32_t blk = 0;              // blocks so far
            uint32_t r = 0, ph = 0;        // group of the (FP8 key or) value ring; parity of the keys' or values' ring
            auto issue_qk = [&](bool last) -> bool {
                if constexpr (FP8) {
                    // the fifth tile in two parts, both times Q's last chunk, and tile 3 into the last
                    // accumulator; tiles 0 to 2 into their own
#pragma unroll 1
                    for (int g = 0; g < 5; ++g) {
                        const int tile = g < 2 ? 3 : g - 2;
                        // the block before's scores have been read: of accumulator 3, of the others
                        if (g == 0 || g == 2) {
                            if (!elected_wait(el, &m->s_empty[g >> 1], (blk & 1) ^ 1, abort, wlim)) return false;
                            tc_fence_after();
                        }
                        if (!elected_wait(el, &m->k_full[r], ph, abort, wlim)) return false;
                        const uint32_t d = tm_s + 64 * tile;
                        const uint64_t kd = k_desc + r * (Cfg::FGROUP / 16);
                        const uint64_t qd = q_desc + (g == 0 ? 8 : 2 * tile) * 512;
                        const uint32_t step = g == 0 ? 0 : 512;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (el)
                                umma_bf16_2cta(d, qd + ((j >> 2) * step + (j & 3) * 2), kd + ((j >> 2) * 512 + (j & 3) * 2),
                                               Cfg::idesc_qk(F16), j != 0 || g == 1);
                        if (el) umma_commit_2cta(&m->k_empty[r], 3);
                        if (el && (g == 1 || g == 4)) umma_commit_2cta(&m->s_full[g >> 2], 3);
                        if (++r == Cfg::FKRING) {
                            r = 0;
                            ph ^= 1;
                        }
                    }
                } else {
                    // scores of this buffer's block before have been read
                    if (!elected_wait(el, &m->s_empty[blk & 1], ((blk >> 1) & 1) ^ 1, abort, wlim)) return false;
                    tc_fence_after();
                    const uint32_t d = tm_s + (blk & 1) * 64;
#pragma unroll 1
                    for (int g = 0; g < (COPY ? 2 : 1) * Cfg::KRING; ++g) {
                        const int kr = g % Cfg::KRING;
                        if (!elected_wait(el, &m->k_full[kr], ph, abort, wlim)) return false;
                        const uint32_t base = kr * (Cfg::KGROUP / 16);   // of Q's chunks as well: 8192 bytes each
#pragma unroll
                        for (int j = 0; j < 12; ++j)
                            if (el) {
                                const uint32_t off = base + (j >> 2) * 512 + (j & 3) * 2;
                                umma_bf16_2cta(d, q_desc + off, k_desc + off, Cfg::idesc_qk(F16), (g | j) != 0);
                            }
                        if (el) umma_commit_2cta(&m->k_empty[kr], 3);
                        if (kr == Cfg::KRING - 1) ph ^= 1;
                    }
                    if (el) umma_commit_2cta(&m->s_full[blk & 1], 3);
                }
                if (last && el) umma_commit_2cta(&m->q_empty, 3);
                return true;
            };
            auto issue_pv = [&](int ngroups, bool first, bool last) -> bool {
                const uint32_t pb = FP8 ? 0u : blk & 1;
                if (!elected_wait(el, &m->p_full[pb], (FP8 ? blk : blk >> 1) & 1, abort, wlim)) return false;
                tc_fence_after();
                const uint64_t pd = p_desc + pb * (Cfg::P_BYTES / 16);
#pragma unroll 1
                for (int g = 0; g < ngroups; ++g) {
                    if (!elected_wait(el, &m->v_full[r], ph, abort, wlim)) return false;
                    const uint64_t vd = v_desc + r * (Cfg::VGROUP / 16);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int s16 = 0; s16 < 2; ++s16)
                            if (el)        // A = P [64 rows x 16 positions] K-major
                                umma_bf16_2cta(tm_o + h * 128, pd + ((g >> 1) * 512 + (g & 1) * 4 + s16 * 2),
                                               vd + (h * 512 + s16 * 128), Cfg::idesc_pv(F16), g > 0 || s16 > 0 || !first);
                    if (el) umma_commit_2cta(&m->v_empty[r], 3);
                    if (++r == (FP8 ? Cfg::FVRING : Cfg::VRING)) {
                        r = 0;
                        ph ^= 1;
                    }
                }
                if (el) umma_commit_2cta(&m->p_empty[pb], 3);
                if (last && el) umma_commit_2cta(&m->o_full, 3);
                return true;
            };
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
                const int nb = __shfl_sync(0xffffffffu, sg.k1 - sg.k0, 0);
                // only the segment's last block can have positions that no row sees
                const int end_groups = __shfl_sync(0xffffffffu, chunk_block(sg, sg.k1 - 1).ngroups, 0);
                if (qk) ok = elected_wait(el, &m->q_full, ns & 1, abort, wlim);
                // O of the segment before must have been read by both epilogues
                else if (ns > 0) ok = elected_wait(el, &m->o_empty, (ns - 1) & 1, abort, wlim);
                for (int i = 0; ok && i < nb; ++i, ++blk)
                    ok = qk ? issue_qk(i + 1 == nb) : issue_pv(i + 1 == nb ? end_groups : Cfg::VGROUPS, i == 0, i + 1 == nb);
            }
            volatile int no_abort = 0;
            if (el) {
                umma_commit_2cta(&m->drain[qk ? 0 : 1], 1);
                mbar_spin(&m->drain[qk ? 0 : 1], 0, &no_abort, wlim);
            }
            __syncwarp();
            if (!ok) *abort = 1;
        }
    } else {
        // ---------------------------------------------------------------- softmax + epilogue
        // 2 * PARTS threads share a row: NP positions of a block each, and VC value columns each in
        // the end.
        constexpr int PARTS = SMW / 4, SMT = 32 * SMW, NP = 64 / PARTS, VC = 256 / PARTS;
        const int L = threadIdx.x & 127;             // TMEM lane
        const int part = threadIdx.x >> 7;
        const int hl = L & 63;                       // row of this CTA's 64
        const int half = L >> 6;
        const int rr = 64 * (int)crank + hl;         // row of the tile
        const int p0 = 64 * half + NP * part;        // first position of this thread in a block
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tm_mine = tm_o + lane_off + VC * part;
        const int col0 = 256 * half + VC * part;     // first of this thread's value columns
        // the row's values of all its threads; `x` of every thread is out before any is read
        auto exchange = [&](float x, float (&of)[2 * PARTS]) {
            s_xm[128 * part + L] = x;
            named_bar_sync(1, SMT);
#pragma unroll
            for (int i = 0; i < 2 * PARTS; ++i) of[i] = s_xm[hl + 64 * i];
            named_bar_sync(1, SMT);
        };
        auto row_sum = [&](float x) -> float {
            float of[2 * PARTS];
            exchange(x, of);
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < 2 * PARTS; i += 2) sum += of[i] + of[i + 1];
            return sum;
        };
        uint32_t blk = 0;
        bool ok = true;
        // Every exit decision of these threads is taken together (votes carried
        // by named barriers), so the named barriers always match.
        for (int ns = 0;; ++ns) {
            const int sr = ns % Cfg::NSEG;
            const bool there = warp_wait(&m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim);
            ok = named_bar_and(1, SMT, ok && there);
            if (!ok) break;
            const TileRun sg = m->seg[sr];
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->seg_empty[sr]);
            if (sg.b < 0) break;
            const bool real = rr < sg.nrows;
            const int tok = sg.tok + (sg.head + rr) / p.H;
            // positions this row sees (rows behind the tile's last hold other rows' queries:
            // computed and dropped)
            const int see = real ? sg.c + tok + 1 : sg.see;
            const int32_t* table = p.block_table + (int64_t)sg.b * p.max_blocks;
            auto page_ok = [&](int k) -> bool { return FP8 || chunk_page(p, sg, table, 2 * k + half) != -2; };
            float c_row = p.scale_log2;                  // scores in log2 units
            if constexpr (F16) {
                ok = warp_wait(&m->q_land, ns & 1, abort, wlim);
                ok = named_bar_and(1, SMT, ok);
                if (!ok) break;
                // This row's 72 pieces of 16 bytes, shared out over its threads (in an order that spreads
                // the lanes over the banks): the largest magnitude, then fp16 of value * 2^(13 - E).
                constexpr int PIECES = 36 / PARTS;
                const int share = 2 * part + half;
                auto piece = [&](int i) -> uint4* {
                    const int j = PIECES * share + i;
                    return reinterpret_cast<uint4*>(s_q + (j >> 3) * 8192 + hl * 128 + (((j + hl) & 7) << 4));
                };
                uint32_t top = 0;                        // bf16 magnitudes compare as integers
#pragma unroll 1
                for (int i = 0; i < PIECES; ++i) {
                    const uint4 v = *piece(i);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        top = max(top, w[e] & 0x7FFFu);
                        top = max(top, (w[e] >> 16) & 0x7FFFu);
                    }
                }
                float of[2 * PARTS];
                exchange(__uint_as_float(top << 16), of);    // (NaN: above infinity as an integer)
#pragma unroll
                for (int e = 0; e < 2 * PARTS; ++e) top = max(top, __float_as_uint(of[e]) >> 16);
                int E = (int)(top >> 7) - 127;
                E = E < -100 ? -100 : E > 127 ? 127 : E;
                const float down = __uint_as_float((uint32_t)(13 - E + 127) << 23);
                c_row *= __uint_as_float((uint32_t)(E - 13 + 127) << 23);
#pragma unroll 1
                for (int i = 0; i < PIECES; ++i) {
                    const uint4 v = *piece(i);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 h = __floats2half2_rn(__uint_as_float(w[e] << 16) * down,
                                                            __uint_as_float(w[e] & 0xFFFF0000u) * down);
                        o[e] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    *piece(i) = make_uint4(o[0], o[1], o[2], o[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_leader(&m->q_full, crank);
            }
            // (the copy) the factor of this thread's page, one block ahead
            auto page_factor = [&](int k, float old) -> float {
                const int page = 2 * k + half;
                return page * kPage < sg.see ? __ldg(p.page_scale + (int64_t)sg.b * p.staged + page) : old;
            };
            bool next_ok = page_ok(sg.k0);
            float next_f = COPY ? page_factor(sg.k0, 1.0f) : 1.0f;
            float mrun = -INFINITY, lrun = 0.0f, lfull = 0.0f;
            for (int k = sg.k0; k < sg.k1; ++k, ++blk) {
                const uint32_t b = FP8 ? 0u : blk & 1, u = (FP8 ? blk : blk >> 1) & 1;
                bool this_ok = next_ok;
                const ChunkScales& rec = s_rec[blk % Cfg::NREC];
                const float fk = next_f;
                if (k + 1 < sg.k1) {
                    next_ok = page_ok(k + 1);
                    if (COPY) next_f = page_factor(k + 1, fk);
                }
                bool got = ok && (FP8 ? warp_wait(&m->rec_full[blk % Cfg::NREC], (blk / Cfg::NREC) & 1, abort, wlim)
                                      : warp_wait(&m->s_full[b], u, abort, wlim));
                float2 sv[NP / 2];
                float mx = -INFINITY;
                if constexpr (FP8) {
                    // the accumulators in the order in which they are made: 3, then 0, 1 and 2
                    this_ok = rec.ok[half] != 0;
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i) sv[i] = make_float2(0.0f, 0.0f);
#pragma unroll 1
                    for (int i4 = 0; got && i4 < 4; ++i4) {
                        const int t = (i4 + 3) & 3;
                        if (i4 < 2) got = warp_wait(&m->s_full[i4], blk & 1, abort, wlim);
                        if (got) {
                            uint32_t a[NP];
                            tc_fence_after();
                            tmem_ld32(tm_s + lane_off + 64 * t + NP * part, a);
                            tmem_wait_ld();
                            tc_fence_before();
                            if (i4 == 0 || i4 == 3) {
                                __syncwarp();
                                if (lane == 0) arrive_leader(&m->s_empty[i4 == 3], crank);
                            }
                            const float4* f4 = reinterpret_cast<const float4*>(&rec.f[t][p0]);
#pragma unroll
                            for (int i = 0; i < NP; i += 4) {
                                const float4 f = f4[i / 4];
                                sv[i / 2] = fma_f32x2(make_float2(__uint_as_float(a[i]), __uint_as_float(a[i + 1])),
                                                      make_float2(f.x, f.y), sv[i / 2]);
                                sv[i / 2 + 1] = fma_f32x2(make_float2(__uint_as_float(a[i + 2]), __uint_as_float(a[i + 3])),
                                                          make_float2(f.z, f.w), sv[i / 2 + 1]);
                            }
                        }
                    }
                }
                if (got) {
                    if constexpr (!FP8) {
                        tc_fence_after();
                        uint32_t a[NP];
                        tmem_ld32(tm_s + lane_off + b * 64 + NP * part, a);
                        tmem_wait_ld();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_leader(&m->s_empty[b], crank);
#pragma unroll
                        for (int i = 0; i < NP; i += 2) {
                            const float2 x = make_float2(__uint_as_float(a[i]), __uint_as_float(a[i + 1]));
                            if constexpr (COPY) {
                                const float c = c_row * fk, l = log2_of_power(fk);
                                sv[i / 2] = fma_f32x2(x, make_float2(c, c), make_float2(l, l));
                            } else {
                                sv[i / 2] = mul_f32x2(x, make_float2(c_row, c_row));
                            }
                        }
                    } else {
                        const float2 l2 = make_float2(rec.log2f[half], rec.log2f[half]);
#pragma unroll
                        for (int i = 0; i < NP / 2; ++i) sv[i] = fma_f32x2(sv[i], make_float2(c_row, c_row), l2);
                    }
                    // positions of this thread that the row sees
                    const int vis = this_ok ? see - (k * Cfg::BLOCK + p0) : 0;
                    if (!__all_sync(0xffffffffu, vis >= NP))
#pragma unroll
                        for (int i = 0; i < NP; i += 2) {
                            sv[i / 2].x = i < vis ? sv[i / 2].x : -INFINITY;
                            sv[i / 2].y = i + 1 < vis ? sv[i / 2].y : -INFINITY;
                        }
#pragma unroll
                    for (int i = 0; i < NP / 2; ++i) mx = fmaxf(mx, fmaxf(sv[i].x, sv[i].y));
                }
                // The reference maximum stays while no thread's scores are above it by more than the limit
                // (one barrier, no exchange); otherwise every row takes its new maximum.
                float muse = mrun;
                bool rescale = false;
                if (!named_bar_and(1, SMT, ok && got && !(mx > mrun + Cfg::lazy(F16)))) {
                    ok = named_bar_and(1, SMT, ok && got);
                    if (!ok) break;
                    float of[2 * PARTS], mnew = -INFINITY;
                    exchange(mx, of);
#pragma unroll
                    for (int i = 0; i < 2 * PARTS; ++i) mnew = fmaxf(mnew, of[i]);
                    rescale = mnew > mrun + Cfg::lazy(F16);      // identical in the threads of a row
                    if (rescale) muse = mnew - Cfg::drop(F16);
                }
                const float base = muse == -INFINITY ? 0.0f : muse;   // (nothing seen yet: 2^-inf)
                uint32_t pk[NP / 2];
                float2 rounded = make_float2(0.0f, 0.0f), full = rounded;
#pragma unroll
                for (int i = 0; i < NP / 2; ++i) {
                    const float2 x = add_f32x2(sv[i], make_float2(-base, -base));
                    const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    // O is divided by the sum of the rounded weights that the MMA multiplies (their
                    // roundings cancel in part); lse takes the sum before rounding.  fp16 weights
                    // divide by that one as well: divided by a small F, the rounding of a
                    // weight that is subnormal in fp16 would count in the sum as it does not in O.
                    if constexpr (F16) {
                        const __half2 h = __floats2half2_rn(e.x, e.y);
                        pk[i] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        pk[i] = pack_bf16(e.x, e.y);
                        rounded = add_f32x2(rounded, make_float2(__uint_as_float(pk[i] << 16), __uint_as_float(pk[i] & 0xFFFF0000u)));
                    }
                    full = add_f32x2(full, e);
                }
                float sum = full.x + full.y;
                if constexpr (COPY) sum /= fk;
                if constexpr (FP8) {
                    sum *= rec.inv[half];
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&m->rec_empty[blk % Cfg::NREC]);
                }
                // weight buffer b is free once P.V of block blk - 2 (FP8: blk - 1) completed
                ok = warp_wait(&m->p_empty[b], u ^ 1, abort, wlim);
                float f = 1.0f;
                const bool need = rescale && k > sg.k0;
                if (need) f = fast_exp2(mrun - muse);
                if (ok && __any_sync(0xffffffffu, need)) {
                    // O at rest: P.V of the block before has completed.  TMEM loads and stores are
                    // warp-wide: lanes whose row keeps its max scale by 1.
                    if (!FP8) ok = warp_wait(&m->p_empty[b ^ 1], ((blk - 1) >> 1) & 1, abort, wlim);
                    if (ok) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < VC; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tm_mine + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(tm_mine + c0, o);
                        }
                        tmem_wait_st();
                    }
                }
                lfull = fmaf(lfull, f, sum);
                lrun = F16 ? lfull : fmaf(lrun, f, rounded.x + rounded.y);
                mrun = muse;
                if (ok) {
                    // P row hl, chunk of this half: 16-byte pieces of a 128-byte row (128-byte swizzle)
                    uint8_t* prow = s_p + b * Cfg::P_BYTES + half * 8192 + hl * 128;
#pragma unroll
                    for (int q = 0; q < NP / 8; ++q)
                        *reinterpret_cast<uint4*>(prow + (((uint32_t)(NP / 8 * part + q) ^ (uint32_t)(hl & 7)) << 4)) =
                            make_uint4(pk[4 * q], pk[4 * q + 1], pk[4 * q + 2], pk[4 * q + 3]);
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader(&m->p_full[b], crank);
                } else {
                    *abort = 1;          // the vote of the next barrier ends the loop in every warp
                }
            }
            // ------------------------------------------------------------ epilogue of a segment
            const bool ofull = ok && warp_wait(&m->o_full, ns & 1, abort, wlim);
            ok = named_bar_and(1, SMT, ofull);
            if (!ok) break;
            const float ltot = row_sum(lrun), lft = F16 ? ltot : row_sum(lfull);
            tc_fence_after();
            const bool empty = ltot == 0.0f;   // the row saw nothing here
            const int64_t row = (int64_t)sg.row0 + rr;
            const float inv = empty ? 0.0f : 1.0f / ltot;
            uint8_t* sl = p.part + Cfg::HEAD_BYTES +
                          ((int64_t)(2 * pair + (sg.part == 1 ? 1 : 0)) * 2 + crank) * Cfg::PART_BYTES;
#pragma unroll 1
            for (int c0 = 0; c0 < VC; c0 += 32) {
                uint32_t o[32];
                tmem_ld32(tm_mine + c0, o);
                tmem_wait_ld();
                if (!real) continue;
                if (empty)                     // O was never written, or holds 0 x anything
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                if (sg.part == 0) {
                    uint4* dst = reinterpret_cast<uint4*>(p.out + row * kDv + col0 + c0);
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[i + e]) * inv;
                        dst[i / 8] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                pack_bf16(v[6], v[7]));
                    }
                } else {
                    uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<float*>(sl) + hl * 512 + col0 + c0);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) __stcg(dst + i / 4, make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
                }
            }
            if (half == 0 && part == 0 && real) {
                if (sg.part != 0)
                    __stcg(reinterpret_cast<float4*>(sl + Cfg::PART_O) + hl,
                           make_float4(empty ? -INFINITY : mrun, ltot, lft, 0.0f));
                else if (p.lse)
                    p.lse[row] = empty ? -INFINITY : (mrun + log2f(lft)) * 0.69314718055994531f;
            }
            // O has been read: the next segment's first P.V may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_leader(&m->o_empty, crank);
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
    if (warp == QK_WARP) {
        tc_fence_after();
        tmem_dealloc_2cta(tmem_base, Cfg::TMEM_COLS);
    }
    if (threadIdx.x == 0 && m->abort) atomicCAS(p.status, 0u, (uint32_t)kStTimeout);
}

// Merge of the tiles whose blocks were spread over several pairs.  Split s of the
// tile that starts in pair x is pair x + s's; with m_s its running maximum (log2
// units), l_s and e_s its sums of weights,
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s,
//   lse = (M + log2 sum_s 2^(m_s - M) e_s) ln 2,  M = max m_s,
// added up in a fixed order.  The rows of all such tiles form one list (a scan over
// the pairs' headers), shared out evenly; four warps take a row, 128 columns each,
// with eight splits' loads in flight per lane.  Where there is a block for every row,
// all of its warps take that row, a quarter of the splits each, joined in shared memory (a
// tile of few rows may have as many splits as there are pairs, and waiting for them
// one by one took 22 us; with four warps a row one token of 16 heads at 4K took 17.4 us, at
// 8K 25.5, one of 128 heads at 16K 34.8; with a block a row 16.6, 18.6 and 26.2).
__global__ void __launch_bounds__(ChunkCfg::COMBINE_THREADS, 1) chunk_combine_kernel(const __grid_constant__ ChunkParams p,
                                                                                     int np) {
    using Cfg = ChunkCfg;
    constexpr int QUARTERS = Cfg::COMBINE_THREADS / 128;
    __shared__ int s_first[Cfg::MAX_PAIRS + 1];          // rows of the pairs before
    __shared__ int4 s_head[Cfg::MAX_PAIRS];
    __shared__ int s_sum[Cfg::COMBINE_THREADS / 32];
    __shared__ float4 s_acc[QUARTERS][128];
    griddep_wait();
    const int lane = (int)(threadIdx.x & 31), warp = (int)(threadIdx.x >> 5);
    int4 h = make_int4(0, 0, 0, 0);
    if ((int)threadIdx.x < np) h = __ldcg(reinterpret_cast<const int4*>(p.part) + threadIdx.x);
    const int mine = h.z >= 2 ? h.y : 0;
    int x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s_sum[w];
    if ((int)threadIdx.x < Cfg::MAX_PAIRS) {
        s_first[threadIdx.x + 1] = before + x;
        s_head[threadIdx.x] = h;
    }
    if (threadIdx.x == 0) s_first[0] = 0;
    __syncthreads();
    const int rows = s_first[Cfg::MAX_PAIRS];
    constexpr int PER = Cfg::MAX_PAIRS / 32;
    const bool whole = rows <= (int)gridDim.x;           // a block takes a row
    const int per = whole ? 1 : QUARTERS, quarter = warp / 4;
    for (int i = (int)blockIdx.x * per + (whole ? 0 : quarter); i < rows; i += (int)gridDim.x * per) {
        int lo = 0, hi = Cfg::MAX_PAIRS - 1;             // the pair whose rows hold i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_first[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        const int row = i - s_first[lo], S = s_head[lo].z;
        const int64_t out_row = (int64_t)s_head[lo].x + row;
        const int crank = row >> 6, hl = row & 63;
        auto slot = [&](int s) -> const uint8_t* {
            return p.part + Cfg::HEAD_BYTES + ((int64_t)(2 * (lo + s) + (s == 0 ? 1 : 0)) * 2 + crank) * Cfg::PART_BYTES;
        };
        float w[PER], l = 0.0f, e = 0.0f, M = -INFINITY;
        float4 st[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int s = lane + 32 * j;
            st[j] = s < S ? __ldcg(reinterpret_cast<const float4*>(slot(s) + Cfg::PART_O) + hl)
                          : make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
            M = fmaxf(M, st[j].x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            w[j] = st[j].x == -INFINITY ? 0.0f : exp2f(st[j].x - M);
            l += w[j] * st[j].y;
            e += w[j] * st[j].z;
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            l += __shfl_xor_sync(0xffffffffu, l, d);
            e += __shfl_xor_sync(0xffffffffu, e, d);
        }
        float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const int col = 128 * (warp & 3) + 4 * lane;
#pragma unroll
        for (int j = 0; j < PER; ++j)
#pragma unroll 1
            for (int g = whole ? 8 * quarter : 0; g < 32 && 32 * j + g < S; g += whole ? 8 * QUARTERS : 8) {
                float4 v[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (32 * j + g + q < S)
                        v[q] = __ldcg(reinterpret_cast<const float4*>(
                            reinterpret_cast<const float*>(slot(32 * j + g + q)) + hl * 512 + col));
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float ws = __shfl_sync(0xffffffffu, w[j], g + q);
                    if (32 * j + g + q < S && ws != 0.0f) {
                        acc.x = fmaf(ws, v[q].x, acc.x);
                        acc.y = fmaf(ws, v[q].y, acc.y);
                        acc.z = fmaf(ws, v[q].z, acc.z);
                        acc.w = fmaf(ws, v[q].w, acc.w);
                    }
                }
            }
        if (whole) {
            __syncthreads();                             // (the row before has been read)
            s_acc[quarter][32 * (warp & 3) + lane] = acc;
            __syncthreads();
            if (quarter > 0) continue;
#pragma unroll
            for (int q = 1; q < QUARTERS; ++q) {
                const float4 o = s_acc[q][32 * (warp & 3) + lane];
                acc.x += o.x;
                acc.y += o.y;
                acc.z += o.z;
                acc.w += o.w;
            }
        }
        const bool empty = l == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / l;
        *reinterpret_cast<uint2*>(p.out + out_row * kDv + col) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if ((warp & 3) == 0 && lane == 0 && p.lse)
            p.lse[out_row] = empty ? -INFINITY : (M + log2f(e)) * 0.69314718055994531f;
    }
}

}  // namespace dsa
