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
// issued by one thread of CTA 0):
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
// of 128 heads sits at the ridge of HBM and tensor rate.
//
// Masked positions.  Scores past a row's own position are replaced, not
// multiplied.  In P.V a weight of zero still multiplies the value row, so rows
// that nobody in the tile sees (the tail of the last page, which may hold
// anything, NaN included) are overwritten with zeros in shared memory, and
// non-finite rows that only some of the tile's tokens see are zeroed too (the
// tokens that see one have a non-finite score already).  Only the slots at the
// tile's causal edge take this path (the "fixer" warp).
//
// Roles per CTA (448 threads):
//   warps 0-7   softmax and epilogue (warps w and w + 4 share TMEM lanes 32(w%4)..;
//               lane L: row 64c + L%64, positions 64*(L/64).. of a block)
//   warp 8      TMEM allocation; CTA 0: issues the score MMAs
//   warp 9      CTA 0: issues the value MMAs
//   warps 10, 11  loads of keys, of values
//   warp 12     segments (runs of one tile's blocks) and the loads of Q
//   warp 13     fixer
#pragma once
#include "common.h"
#include "pair.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

namespace dsa {

struct ChunkCfg {
    static constexpr int ROWS = 128;                    // (token, head) rows of a tile
    static constexpr int BLOCK = 128;                   // positions of a block (two pages)
    static constexpr int KCH = 9;                       // 64-column chunks of a latent row
    static constexpr int KRING = 3;                     // groups of keys (64 rows x 3 chunks) that are kept
    static constexpr int kgroups(bool f16) { return f16 ? 6 : 3; }   // groups that make a block
    static constexpr int KGROUP = 3 * 8192;
    static constexpr int VGROUPS = 4;                   // groups of a block's values: 32 rows x 4 chunks (this CTA's)
    static constexpr int VRING = 3;                     // groups that are kept
    static constexpr int VGROUP = 4 * 4096;
    static constexpr int Q_BYTES = KCH * 64 * 128;      // this CTA's 64 rows
    static constexpr int P_BYTES = 64 * BLOCK * 2;      // [64 rows x 128 positions] bf16: two 64-position chunks
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + Q_BYTES;
    static constexpr int OFF_K = OFF_P + 2 * P_BYTES;
    static constexpr int OFF_V = OFF_K + KRING * KGROUP;
    static constexpr int OFF_XM = OFF_V + VRING * VGROUP;   // exchange between the threads of a row
    static constexpr int OFF_MISC = OFF_XM + 256 * 4;
    static constexpr int MISC_BYTES = 1024;
    static constexpr int SMEM = 1024 + OFF_MISC + MISC_BYTES;
    static constexpr int SOFTMAX_WARPS = 8;
    static constexpr int QK_WARP = 8, PV_WARP = 9, KEY_WARP = 10, VALUE_WARP = 11, SEG_WARP = 12, FIX_WARP = 13;
    static constexpr int THREADS = 448;
    // A row's reference (a maximum minus DROP) is replaced once a score exceeds it by more than LAZY.
    // bf16 weights and fp32 sums are floating point, so a reference below the maximum costs no
    // precision, and 2^32 (2^52 for the sums of a million weights) is far from fp32's range; a
    // replacement waits for the P.V in flight.  fp16 weights end at 2^16 and lose bits below
    // 2^-14: references seven below the maximum keep them in [2^-14, 2^15] down to 2^-21 of the
    // largest weight, and to 2^-32 of it with an absolute error.
    static constexpr float lazy(bool f16) { return f16 ? 15.0f : 32.0f; }
    static constexpr float drop(bool f16) { return f16 ? 7.0f : 0.0f; }
    static constexpr int NSEG = 4;                      // segment ring
    static constexpr int TMEM_COLS = 512;               // O: [0, 256), two score buffers of 64 from column 256
    // fp16 operands: the bf16 descriptor without its two operand-format bits
    static constexpr uint32_t BF16_BITS = (1u << 7) | (1u << 10);
    static constexpr uint32_t idesc_qk(bool f16) { return idesc_bf16_f32(128, BLOCK, false, false) & ~(f16 ? BF16_BITS : 0u); }
    static constexpr uint32_t idesc_pv(bool f16) { return idesc_bf16_f32(128, 256, false, true) & ~(f16 ? BF16_BITS : 0u); }
    // partial result of (pair, side, CTA): O [64 rows][512] fp32, then (m, sum, sum for lse, -) per row.
    // Side 1: the pair holds the tile's first blocks; side 0: later ones.
    static constexpr int64_t PART_O = 64 * 512 * 4;
    static constexpr int64_t PART_BYTES = PART_O + 64 * 16;
    static constexpr int64_t HEAD_BYTES = 2048;         // one int4 per pair: the tile that starts there and ends in a later pair
    static constexpr int MAX_PAIRS = 128;                // the merge keeps four splits per lane
    static constexpr int COMBINE_THREADS = 256;         // at least MAX_PAIRS
};
static_assert(ChunkCfg::SMEM <= 232448, "shared memory exceeds the per-CTA limit");
static_assert(ChunkCfg::OFF_P % 1024 == 0 && ChunkCfg::OFF_K % 1024 == 0 && ChunkCfg::OFF_V % 1024 == 0, "swizzled operands need 1024-byte alignment");
static_assert(ChunkCfg::COMBINE_THREADS >= ChunkCfg::MAX_PAIRS, "one thread per header");
static_assert(ChunkCfg::MAX_PAIRS * 16 <= ChunkCfg::HEAD_BYTES, "one header per pair");

using ChunkTiles = TileList<ChunkCfg::ROWS, ChunkCfg::BLOCK>;

struct ChunkParams : ListParams {
    uint16_t* out;            // [T, H, 512] bf16 bits
    float* lse;               // [T, H] or null
    uint8_t* part;            // headers, then partial results
    uint32_t* status;         // status word; words 1-2 hold the test hooks
    const float* page_scale;  // [B, staged] the copy's power-of-two factor of each page
    float scale_log2;         // sm_scale * log2(e)
};

struct ChunkMisc {
    uint64_t k_full[ChunkCfg::KRING];   // (CTA 0) the key group is ready in both CTAs
    uint64_t k_empty[ChunkCfg::KRING];  // its MMAs have completed
    uint64_t v_full[ChunkCfg::VRING];   // (CTA 0) the value group is ready in both CTAs
    uint64_t v_empty[ChunkCfg::VRING];
    uint64_t v_peer[ChunkCfg::VRING];     // (CTA 0) CTA 1's fixer is done with the group
    uint64_t v_land[ChunkCfg::VRING];   // the group has landed, for the fixer to look at
    uint64_t q_full;                      // (CTA 0) Q of both CTAs
    uint64_t q_land;                      // (fp16) this CTA's Q, still bf16
    uint64_t q_empty;
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t o_full, o_empty, drain[2];
    uint64_t seg_full[ChunkCfg::NSEG], seg_empty[ChunkCfg::NSEG];
    TileRun seg[ChunkCfg::NSEG];
    uint64_t wait_ns;
    ShareStart start;
    int64_t sums[ChunkCfg::THREADS / 32];
    uint32_t tmem_base;
    int abort;
    uint32_t inject;
};
static_assert(sizeof(ChunkMisc) <= ChunkCfg::MISC_BYTES, "misc block exceeds its slot");

// The 32-position groups of a block that the value product runs over.
struct ChunkBlock {
    int ngroups;              // 32-position groups that some row sees (1..4)
    int fix_from;             // first group that the fixer looks at (ngroups: none)
};
__device__ __forceinline__ ChunkBlock chunk_block(const TileRun& s, int k) {
    ChunkBlock r;
    const int left = s.see - k * ChunkCfg::BLOCK;          // positions of the block that some row sees
    r.ngroups = left >= ChunkCfg::BLOCK ? 4 : left > 0 ? (left + 31) / 32 : 0;
    const int all = s.see_all - k * ChunkCfg::BLOCK;       // ... that every row sees
    r.fix_from = all <= 0 ? 0 : all / 32;
    if (r.fix_from > r.ngroups) r.fix_from = r.ngroups;
    return r;
}

// F16: the cache is the fp16 copy of an FP8 cache (latent.cu), and Q is
// brought to fp16 in shared memory: both operands of an MMA have one type, and
// bf16 would round the products of codes and scales eight times as far.  A row of
// the copy holds the 576 rounded values and what their rounding left out; the
// scores take both (twice the score MMAs and key loads: with the rounded values
// alone lse was off by 6e-6 of itself, with both by 3e-7), the value product the
// first.  Powers of two keep the values in fp16's range: one per row of Q,
// one per page f_s of the copy.  With t_s = S_s + log2 f_s the weights that
// multiply the copy's rows are P_s f_s = 2^(t_s - m), so the reference m follows
// t, and the sums of weights are those of 2^(t_s - m) / f_s.
template <bool F16>
__global__ void __launch_bounds__(ChunkCfg::THREADS, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using Cfg = ChunkCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_shared(smem_raw, 1024);
    uint8_t* s_q = smem + Cfg::OFF_Q;
    uint8_t* s_p = smem + Cfg::OFF_P;
    uint8_t* s_k = smem + Cfg::OFF_K;
    uint8_t* s_v = smem + Cfg::OFF_V;
    float* s_xm = reinterpret_cast<float*>(smem + Cfg::OFF_XM);
    ChunkMisc* m = reinterpret_cast<ChunkMisc*>(smem + Cfg::OFF_MISC);
    volatile int* abort = &m->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    int np = (int)(gridDim.x >> 1);
    const int pair = (int)(blockIdx.x >> 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::KRING; ++i) {
            mbar_init(&m->k_full[i], 1);    // CTA 0's loader, for both CTAs
            mbar_init(&m->k_empty[i], 1);
        }
        for (int i = 0; i < Cfg::VRING; ++i) {
            mbar_init(&m->v_full[i], 1);    // CTA 0's loader or fixer, for both CTAs
            mbar_init(&m->v_peer[i], 1);
            mbar_init(&m->v_empty[i], 1);
            mbar_init(&m->v_land[i], 1);
        }
        mbar_init(&m->q_full, F16 ? 2 * Cfg::SOFTMAX_WARPS : 2);
        mbar_init(&m->q_land, 1);
        mbar_init(&m->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->s_empty[i], 2 * Cfg::SOFTMAX_WARPS);   // those of both CTAs
            mbar_init(&m->p_full[i], 2 * Cfg::SOFTMAX_WARPS);
            mbar_init(&m->p_empty[i], 1);
            mbar_init(&m->drain[i], 1);
        }
        mbar_init(&m->o_full, 1);
        mbar_init(&m->o_empty, 2 * Cfg::SOFTMAX_WARPS);
        for (int i = 0; i < Cfg::NSEG; ++i) {
            mbar_init(&m->seg_full[i], 1);
            mbar_init(&m->seg_empty[i], Cfg::SOFTMAX_WARPS + (crank == 0 ? 5 : 3));   // loading and fixer warps; CTA 0: the issuers too
        }
        m->abort = 0;
        m->start.b = -1;
        fence_mbar_init();
    }
    if (warp == Cfg::QK_WARP) {
        tmem_alloc_2cta(&m->tmem_base, Cfg::TMEM_COLS);
        tmem_relinquish_2cta();
    }
    if (warp == Cfg::SEG_WARP && lane == 0) {
        prefetch_tmap(&tm_q);
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
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
    const uint32_t tm_s = tmem_base + 256;      // score buffers, 64 columns each
    const uint64_t wlim = m->wait_ns;

    // ---------------------------------------------------------------- this pair's share of the list
    int64_t g0, g1, total;
    ChunkTiles::share<Cfg::THREADS>(p, pair, np, m->sums, &m->start, p.status, g0, g1, total);

    if (warp == Cfg::SEG_WARP) {
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
    } else if (warp == Cfg::KEY_WARP || warp == Cfg::VALUE_WARP) {
        // ---------------------------------------------------------------- loads of keys, of values
        // The whole warp runs the schedule and one elected lane acts, so that addresses and
        // coordinates stay in uniform registers (per-lane values would have to be moved there for
        // every copy).  CTA 0 announces the bytes of both CTAs (both see the same page ids), so
        // that CTA 1 only issues its copies.
        const bool keys = warp == Cfg::KEY_WARP;
        const bool el = elect_one();
        // test hook: the second CTA never loads
        bool ok = !(crank == 1 && (m->inject & 4u));
        bool bad = false;
        uint32_t r = 0, ph = 1;            // group of the (value) ring and the parity that its `empty` waits for
        const uint32_t k_lead = mapa_shared(smem_u32(&m->k_full[0]), 0), v_lead = mapa_shared(smem_u32(&m->v_full[0]), 0);
        TileRun sg = {};
        const int32_t* table = nullptr;
        auto page_id = [&](int page) -> int {          // -1: nobody sees the page; -2: a bad id
            if (page >= p.max_blocks || page * kPage >= sg.see) return -1;
            const int id = __ldg(table + page);
            return id >= 0 && id < p.num_blocks ? (p.staged ? sg.b * p.staged + page : id) : -2;
        };
        auto load_keys = [&](int id0, int id1) -> bool {
            const int id = crank == 0 ? id0 : id1;
            // a page that nobody sees is not loaded: its scores are replaced whatever they are
            const uint32_t bytes = (uint32_t)Cfg::KGROUP * ((id0 >= 0) + (id1 >= 0));
            const bool mine = el && id >= 0;
            const int y = id * kPage;
#pragma unroll 1
            for (int g = 0; g < Cfg::kgroups(F16); ++g) {
                const int kr = g % Cfg::KRING;
                if (!elected_wait(el, &m->k_empty[kr], ph, abort, wlim)) return false;
                if (crank == 0 && el) mbar_arrive_expect_tx(&m->k_full[kr], bytes);
                // (fp16: the small rests first, so that adding them up costs no bits of the sum)
                const int chunk = F16 && g < Cfg::KRING ? 3 * g + 9 : F16 ? 3 * g - 9 : 3 * g;
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
    } else if (warp == Cfg::FIX_WARP) {
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
    } else if (warp == Cfg::QK_WARP || warp == Cfg::PV_WARP) {
        // ---------------------------------------------------------------- MMA issuers (CTA 0)
        // The whole warp runs the schedule and one elected lane issues, so that the operand
        // descriptors stay in uniform registers: 30 cycles per MMA where descriptors kept per
        // lane cost 51 (the MMAs themselves take 32 and 64).  Descriptors differ from a base by
        // multiples of 16 bytes in their low words.
        const bool qk = warp == Cfg::QK_WARP;
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
            uint32_t r = 0, ph = 0;        // group of the value ring; parity of the keys' or values' ring
            auto issue_qk = [&](bool last) -> bool {
                // scores of this buffer's block before have been read
                if (!elected_wait(el, &m->s_empty[blk & 1], ((blk >> 1) & 1) ^ 1, abort, wlim)) return false;
                tc_fence_after();
                const uint32_t d = tm_s + (blk & 1) * 64;
#pragma unroll 1
                for (int g = 0; g < Cfg::kgroups(F16); ++g) {
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
                if (last && el) umma_commit_2cta(&m->q_empty, 3);
                return true;
            };
            auto issue_pv = [&](int ngroups, bool first, bool last) -> bool {
                if (!elected_wait(el, &m->p_full[blk & 1], (blk >> 1) & 1, abort, wlim)) return false;
                tc_fence_after();
                const uint64_t pd = p_desc + (blk & 1) * (Cfg::P_BYTES / 16);
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
                    if (++r == Cfg::VRING) {
                        r = 0;
                        ph ^= 1;
                    }
                }
                if (el) umma_commit_2cta(&m->p_empty[blk & 1], 3);
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
        // Four threads share a row: positions 64 * half + 32 * part .. of a block each, and 128
        // value columns each in the end.
        const int L = threadIdx.x & 127;             // TMEM lane
        const int part = threadIdx.x >> 7;
        const int hl = L & 63;                       // row of this CTA's 64
        const int half = L >> 6;
        const int rr = 64 * (int)crank + hl;         // row of the tile
        const int p0 = 64 * half + 32 * part;        // first position of this thread in a block
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tm_mine = tm_o + lane_off + 128 * part;
        const int col0 = 256 * half + 128 * part;    // first of this thread's value columns
        // the row's value of all four threads combined; `x` of every thread is out before any is read
        auto exchange = [&](float x, float (&of)[4]) {
            s_xm[128 * part + L] = x;
            named_bar_sync(1, 256);
            of[0] = s_xm[hl];
            of[1] = s_xm[hl + 64];
            of[2] = s_xm[hl + 128];
            of[3] = s_xm[hl + 192];
            named_bar_sync(1, 256);
        };
        uint32_t blk = 0;
        bool ok = true;
        // Every exit decision of these 256 threads is taken together (votes carried
        // by named barriers), so the named barriers always match.
        for (int ns = 0;; ++ns) {
            const int sr = ns % Cfg::NSEG;
            const bool there = warp_wait(&m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim);
            ok = named_bar_and(1, 256, ok && there);
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
            auto page_ok = [&](int k) -> bool {
                const int page = 2 * k + half;
                if (page >= p.max_blocks || page * kPage >= sg.see) return true;   // masked by position
                const int id = __ldg(table + page);
                return id >= 0 && id < p.num_blocks;
            };
            float c_row = p.scale_log2;                  // scores in log2 units
            const float* page_scale = nullptr;
            if constexpr (F16) {
                page_scale = p.page_scale + (int64_t)sg.b * p.staged;
                ok = warp_wait(&m->q_land, ns & 1, abort, wlim);
                ok = named_bar_and(1, 256, ok);
                if (!ok) break;
                // This row's 72 pieces of 16 bytes, 18 for each of its threads (in an order that spreads
                // the lanes over the banks): the largest magnitude, then fp16 of value * 2^(13 - E).
                const int quarter = 2 * part + half;
                auto piece = [&](int i) -> uint4* {
                    const int j = 18 * quarter + i;
                    return reinterpret_cast<uint4*>(s_q + (j >> 3) * 8192 + hl * 128 + (((j + hl) & 7) << 4));
                };
                uint32_t top = 0;                        // bf16 magnitudes compare as integers
#pragma unroll 1
                for (int i = 0; i < 18; ++i) {
                    const uint4 v = *piece(i);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        top = max(top, w[e] & 0x7FFFu);
                        top = max(top, (w[e] >> 16) & 0x7FFFu);
                    }
                }
                float of[4];
                exchange(__uint_as_float(top << 16), of);    // (NaN: above infinity as an integer)
                for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(of[e]) >> 16);
                int E = (int)(top >> 7) - 127;
                E = E < -100 ? -100 : E > 127 ? 127 : E;
                const float down = __uint_as_float((uint32_t)(13 - E + 127) << 23);
                c_row *= __uint_as_float((uint32_t)(E - 13 + 127) << 23);
#pragma unroll 1
                for (int i = 0; i < 18; ++i) {
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
            bool next_ok = page_ok(sg.k0);
            float next_f = 1.0f;
            if constexpr (F16)
                if ((2 * sg.k0 + half) * kPage < sg.see) next_f = __ldg(page_scale + 2 * sg.k0 + half);
            float mrun = -INFINITY, lrun = 0.0f, lfull = 0.0f;
            for (int k = sg.k0; k < sg.k1; ++k, ++blk) {
                const uint32_t b = blk & 1, u = (blk >> 1) & 1;
                const bool this_ok = next_ok;
                const float fk = next_f;
                if (k + 1 < sg.k1) {
                    next_ok = page_ok(k + 1);
                    if constexpr (F16)
                        if ((2 * (k + 1) + half) * kPage < sg.see) next_f = __ldg(page_scale + 2 * (k + 1) + half);
                }
                const bool got = ok && warp_wait(&m->s_full[b], u, abort, wlim);
                float sv[32];
                float mx = -INFINITY;
                if (got) {
                    tc_fence_after();
                    uint32_t a[32];
                    tmem_ld32(tm_s + lane_off + b * 64 + 32 * part, a);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader(&m->s_empty[b], crank);
                    // positions of this thread that the row sees
                    const int vis = this_ok ? see - (k * Cfg::BLOCK + p0) : 0;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        sv[i] = F16 ? fmaf(__uint_as_float(a[i]), c_row * fk, log2_of_power(fk)) : __uint_as_float(a[i]) * c_row;
                    if (!__all_sync(0xffffffffu, vis >= 32))
#pragma unroll
                        for (int i = 0; i < 32; ++i) sv[i] = i < vis ? sv[i] : -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, sv[i]);
                }
                // The reference maximum stays while no thread's scores are above it by more than the limit
                // (one barrier, no exchange); otherwise every row takes its new maximum.
                float muse = mrun;
                bool rescale = false;
                if (!named_bar_and(1, 256, ok && got && !(mx > mrun + Cfg::lazy(F16)))) {
                    ok = named_bar_and(1, 256, ok && got);
                    if (!ok) break;
                    float of[4];
                    exchange(mx, of);
                    const float mnew = fmaxf(fmaxf(of[0], of[1]), fmaxf(of[2], of[3]));
                    rescale = mnew > mrun + Cfg::lazy(F16);      // identical in the four threads of a row
                    if (rescale) muse = mnew - Cfg::drop(F16);
                }
                const float base = muse == -INFINITY ? 0.0f : muse;   // (nothing seen yet: 2^-inf)
                uint32_t pk[16];
                float r0 = 0.0f, r1 = 0.0f, f0 = 0.0f, f1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float e0 = fast_exp2(sv[2 * i] - base);
                    const float e1 = fast_exp2(sv[2 * i + 1] - base);
                    // O is divided by the sum of the rounded weights that the MMA multiplies (their
                    // roundings cancel in part); lse takes the sum before rounding.  fp16 weights
                    // divide by that one as well: divided by a small page factor, the rounding of a
                    // weight that is subnormal in fp16 would count in the sum as it does not in O.
                    if constexpr (F16) {
                        const __half2 h = __floats2half2_rn(e0, e1);
                        pk[i] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        pk[i] = pack_bf16(e0, e1);
                        r0 += __uint_as_float(pk[i] << 16);
                        r1 += __uint_as_float(pk[i] & 0xFFFF0000u);
                    }
                    f0 += e0;
                    f1 += e1;
                }
                // weight buffer b is free once P.V of block blk - 2 completed
                ok = warp_wait(&m->p_empty[b], u ^ 1, abort, wlim);
                float f = 1.0f;
                const bool need = rescale && k > sg.k0;
                if (need) f = fast_exp2(mrun - muse);
                if (ok && __any_sync(0xffffffffu, need)) {
                    // O at rest: P.V of the block before has completed.  TMEM loads and stores are
                    // warp-wide: lanes whose row keeps its max scale by 1.
                    ok = warp_wait(&m->p_empty[b ^ 1], ((blk - 1) >> 1) & 1, abort, wlim);
                    if (ok) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < 128; c0 += 32) {
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
                lfull = fmaf(lfull, f, F16 ? (f0 + f1) / fk : f0 + f1);
                lrun = F16 ? lfull : fmaf(lrun, f, r0 + r1);
                mrun = muse;
                if (ok) {
                    // P row hl, chunk of this half: four 16-byte pieces of a 128-byte row (128-byte swizzle)
                    uint8_t* prow = s_p + b * Cfg::P_BYTES + half * 8192 + hl * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint4*>(prow + (((uint32_t)(4 * part + q) ^ (uint32_t)(hl & 7)) << 4)) =
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
            ok = named_bar_and(1, 256, ofull);
            if (!ok) break;
            float of[4];
            exchange(lrun, of);
            const float ltot = (of[0] + of[1]) + (of[2] + of[3]);
            exchange(lfull, of);
            const float lft = (of[0] + of[1]) + (of[2] + of[3]);
            tc_fence_after();
            const bool empty = ltot == 0.0f;   // the row saw nothing here
            const int64_t row = (int64_t)sg.row0 + rr;
            const float inv = empty ? 0.0f : 1.0f / ltot;
            uint8_t* sl = p.part + Cfg::HEAD_BYTES +
                          ((int64_t)(2 * pair + (sg.part == 1 ? 1 : 0)) * 2 + crank) * Cfg::PART_BYTES;
#pragma unroll 1
            for (int c0 = 0; c0 < 128; c0 += 32) {
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
    if (warp == Cfg::QK_WARP) {
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
// added up in split order.  The rows of all such tiles form one list (a scan over
// the pairs' headers), shared out evenly; four warps take a row, 128 columns each,
// with eight splits' loads in flight per lane (a tile of few rows may have as many
// splits as there are pairs, and waiting for them one by one took 22 us).
__global__ void __launch_bounds__(ChunkCfg::COMBINE_THREADS) chunk_combine_kernel(const __grid_constant__ ChunkParams p,
                                                                                  int np) {
    using Cfg = ChunkCfg;
    constexpr int ROWS = Cfg::COMBINE_THREADS / 128;     // rows a block takes at a time
    __shared__ int s_first[Cfg::MAX_PAIRS + 1];          // rows of the pairs before
    __shared__ int4 s_head[Cfg::MAX_PAIRS];
    __shared__ int s_sum[Cfg::COMBINE_THREADS / 32];
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
    for (int i = (int)blockIdx.x * ROWS + warp / 4; i < rows; i += (int)gridDim.x * ROWS) {
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
            for (int g = 0; g < 32 && 32 * j + g < S; g += 8) {
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
        const bool empty = l == 0.0f;
        const float inv = empty ? 0.0f : 1.0f / l;
        *reinterpret_cast<uint2*>(p.out + out_row * kDv + col) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
        if ((warp & 3) == 0 && lane == 0 && p.lse)
            p.lse[out_row] = empty ? -INFINITY : (M + log2f(e)) * 0.69314718055994531f;
    }
}

}  // namespace dsa
