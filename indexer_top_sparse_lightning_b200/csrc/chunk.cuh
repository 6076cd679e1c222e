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
// chunk_combine_kernel.  The list is never stored: the blocks of a sequence's
// first i tiles have a closed form (tile_prefix below).
//
// Per block the pair runs two-CTA tensor-core MMAs (tcgen05 cta_group::2,
// issued by one thread of CTA 0):
//   S = Q.K^T: M = 128 rows (64 per CTA), N = 128 positions (CTA c holds page
//       2k + c), nine K-chunks of 64 columns;
//   O += P.V: M = 128 rows, N = 256 value columns twice (CTA c holds columns
//       128c.. and 256 + 128c.. of both pages), K = 128 positions.
// Both operands come through ONE ring of 8 KB slots filled by one thread in
// the very order in which the MMAs consume them (a 64 x 64 box of keys, or 32
// rows x 128 value columns), across block and tile boundaries: 15 slots keep
// 120 KB per SM in flight, more than a block's worth, with no fixed split
// between keys and values.  S of block k + 1 is computed before P.V of block k,
// so the softmax of one block runs under the products of its neighbours.
// Loads of both CTAs are counted on CTA 0's barriers (the two-CTA form of the
// tiled load), so nobody forwards arrivals.
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
// Roles per CTA (256 threads):
//   warps 0-3   softmax and epilogue (thread L <-> TMEM lane L: row 64c + L%64,
//               positions 64*(L/64).. of a block)
//   warp 4      TMEM allocation; CTA 0: MMA issuer
//   warp 5      loads of keys and values
//   warp 6      segments (runs of one tile's blocks) and the loads of Q
//   warp 7      fixer
#pragma once
#include "common.h"
#include "fp8row.cuh"
#include "pair.cuh"
#include "ptx.cuh"

namespace dsa {

struct ChunkCfg {
    static constexpr int ROWS = 128;                    // (token, head) rows of a tile
    static constexpr int BLOCK = 128;                   // positions of a block (two pages)
    static constexpr int KCH = 9;                       // 64-column chunks of a latent row
    static constexpr int SLOT = 8192;
    static constexpr int NSLOT = 15;
    static constexpr int Q_BYTES = KCH * 64 * 128;      // this CTA's 64 rows
    static constexpr int P_BYTES = 64 * BLOCK * 2;      // [64 rows x 128 positions] bf16: two 64-position chunks
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + Q_BYTES;
    static constexpr int OFF_RING = OFF_P + 2 * P_BYTES;
    static constexpr int OFF_XM = OFF_RING + NSLOT * SLOT;   // partner exchange, two buffers of 128 floats
    static constexpr int OFF_MISC = OFF_XM + 2 * 128 * 4;
    static constexpr int MISC_BYTES = 1024;
    static constexpr int SMEM = 1024 + OFF_MISC + MISC_BYTES;
    static constexpr int THREADS = 256;
    static constexpr int MMA_WARP = 4, LOAD_WARP = 5, SEG_WARP = 6, FIX_WARP = 7;
    static constexpr int NSEG = 4;                      // segment ring
    static constexpr int TMEM_COLS = 512;               // O: [0, 256), two score buffers of 64 from column 256
    static constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, BLOCK, false, false);
    static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, 256, false, true);
    // partial result of (pair, side, CTA): O [64 rows][512] fp32, then (m, sum, sum for lse, -) per row.
    // Side 1: the pair holds the tile's first blocks; side 0: later ones.
    static constexpr int64_t PART_O = 64 * 512 * 4;
    static constexpr int64_t PART_BYTES = PART_O + 64 * 16;
    static constexpr int64_t HEAD_BYTES = 2048;         // one int4 per pair: the tile that starts there and ends in a later pair
    static constexpr int MAX_PAIRS = 128;                // the merge keeps four splits per lane
    static constexpr int COMBINE_THREADS = 256;
};
static_assert(ChunkCfg::SMEM <= 232448, "shared memory exceeds the per-CTA limit");
static_assert(ChunkCfg::OFF_P % 1024 == 0 && ChunkCfg::OFF_RING % 1024 == 0, "swizzled operands need 1024-byte alignment");
static_assert(ChunkCfg::MAX_PAIRS * 16 <= ChunkCfg::HEAD_BYTES, "one header per pair");

struct ChunkParams {
    const int32_t* seq_lens;
    const int32_t* cu_q;
    const int32_t* block_table;
    uint16_t* out;            // [T, H, 512] bf16 bits
    float* lse;               // [T, H] or null
    uint8_t* part;            // headers, then partial results
    uint32_t* status;         // status word; words 1-2 hold the test hooks
    int32_t B, T, H, max_blocks, num_blocks;
    int32_t staged;           // > 0: the cache is a copy by sequence, `staged` pages each
    float scale_log2;         // sm_scale * log2(e)
};

// A run of blocks of one tile.
struct ChunkSeg {
    int32_t b;                // sequence, -1: no more segments
    int32_t row0;             // first (token, head) row of the tile, over the whole batch
    int32_t nrows;            // rows of the tile (up to 128)
    int32_t tok, head;        // token (in its sequence) and head of that row
    int32_t c;                // position of the sequence's first new token
    int32_t k0, k1;           // blocks
    int32_t see_all, see;     // positions below see_all are seen by every row, none at or above see by any
    int32_t part;             // 0: the whole tile; 1: its first blocks; 2: later blocks
    int32_t pad;
};

struct ChunkMisc {
    uint64_t full[ChunkCfg::NSLOT];     // (CTA 0) a slot of both CTAs is ready for the MMAs
    uint64_t empty[ChunkCfg::NSLOT];    // its MMAs have completed
    uint64_t land[ChunkCfg::NSLOT];     // bytes of a slot that the fixer looks at have landed
    uint64_t q_full;                    // (CTA 0) Q of both CTAs
    uint64_t q_empty;
    uint64_t s_full[2], s_empty[2], p_full[2], p_empty[2];
    uint64_t o_full, o_empty, drain;
    uint64_t seg_full[ChunkCfg::NSEG], seg_empty[ChunkCfg::NSEG];
    ChunkSeg seg[ChunkCfg::NSEG];
    uint64_t wait_ns;
    int64_t start_before;               // blocks before the sequence that this pair starts in
    int64_t sums[ChunkCfg::THREADS / 32];
    int32_t start_b;
    uint32_t tmem_base;
    int abort;
    uint32_t inject;
};
static_assert(sizeof(ChunkMisc) <= ChunkCfg::MISC_BYTES, "misc block exceeds its slot");

// ------------------------------------------------------------------ the block list
// One sequence as the list sees it.
struct ChunkSeq {
    int32_t row0, rows;       // its (token, head) rows
    int32_t c, n, len;        // position of its first new token, new tokens, cached length
    int32_t tiles, first;     // tiles; (c * H - 1) / 128, rounded down
    int64_t blocks;           // blocks of all tiles
};

// sum over x < n of floor(x / h)
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t h) {
    const uint32_t q = n / h, r = n % h;
    return (int64_t)h * q * (q > 0 ? q - 1 : 0) / 2 + (int64_t)r * q;
}

// Blocks of the tiles before tile i (i < tiles).  Tile k < tiles - 1 ends with
// row 128(k + 1) - 1, so it sees c + floor((128(k + 1) - 1) / H) + 1 positions,
// in floor((c + floor((128(k + 1) - 1) / H)) / 128) + 1 blocks, which is
// floor((k + 1 + first) / H) + 1 with first = floor((c H - 1) / 128) (nested
// floors of quotients by integers commute).
__device__ __forceinline__ int64_t tile_prefix(const ChunkSeq& s, int H, int i) {
    return (int64_t)i + floor_sum((uint32_t)(i + 1 + s.first), (uint32_t)H) - floor_sum((uint32_t)(1 + s.first), (uint32_t)H);
}
__device__ __forceinline__ int64_t last_tile_blocks(const ChunkSeq& s) { return (s.c + s.n - 1) / ChunkCfg::BLOCK + 1; }

// Sequence b, with sizes that no input can push out of range: tokens past T are
// dropped, a length is cut to the table's (both reported by `ok`).
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int b, bool& ok) {
    ChunkSeq s;
    int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
    const int64_t cap = (int64_t)(p.staged ? p.staged : p.max_blocks) * kPage;
    const int64_t len = __ldg(p.seq_lens + b);
    ok = q0 >= 0 && q1 >= q0 && q1 <= p.T && len <= cap && (q1 == q0 || len >= q1 - q0);
    q0 = q0 < 0 ? 0 : q0 > p.T ? p.T : q0;
    q1 = q1 < q0 ? q0 : q1 > p.T ? p.T : q1;
    s.n = q1 - q0;
    s.len = (int)(len < 0 ? 0 : len > cap ? cap : len);
    if (s.len < s.n) s.n = s.len;             // a sequence shorter than its new tokens: the rest sees nothing
    s.c = s.len - s.n;
    s.row0 = q0 * p.H;
    s.rows = s.n * p.H;
    s.tiles = (s.rows + ChunkCfg::ROWS - 1) / ChunkCfg::ROWS;
    const int64_t ch = (int64_t)s.c * p.H;
    s.first = ch > 0 ? (int)((ch - 1) / ChunkCfg::ROWS) : -1;
    s.blocks = s.tiles > 0 ? tile_prefix(s, p.H, s.tiles - 1) + last_tile_blocks(s) : 0;
    return s;
}

// Sum over the block's threads, the same in all of them; `excl` receives the sum
// of the threads before this one.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sums, int64_t& excl) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
        if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    int64_t total = 0, before = 0;
    for (int w = 0; w < nw; ++w) {
        if (w == warp) before = total;
        total += sums[w];
    }
    excl = before + x - v;
    return total;
}

// The rows at or past this row limit of a block see nothing of it.
struct ChunkBlock {
    int ngroups;              // 32-position groups that some row sees (1..4)
    int fix_from;             // first group that the fixer looks at (ngroups: none)
};
__device__ __forceinline__ ChunkBlock chunk_block(const ChunkSeg& s, int k) {
    ChunkBlock r;
    const int left = s.see - k * ChunkCfg::BLOCK;          // positions of the block that some row sees
    r.ngroups = left >= ChunkCfg::BLOCK ? 4 : left > 0 ? (left + 31) / 32 : 0;
    const int all = s.see_all - k * ChunkCfg::BLOCK;       // ... that every row sees
    r.fix_from = all <= 0 ? 0 : all / 32;
    if (r.fix_from > r.ngroups) r.fix_from = r.ngroups;
    return r;
}

__global__ void __launch_bounds__(ChunkCfg::THREADS, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkParams p, const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
    using Cfg = ChunkCfg;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = align_shared(smem_raw, 1024);
    uint8_t* s_q = smem + Cfg::OFF_Q;
    uint8_t* s_p = smem + Cfg::OFF_P;
    uint8_t* s_ring = smem + Cfg::OFF_RING;
    float* s_xm = reinterpret_cast<float*>(smem + Cfg::OFF_XM);
    ChunkMisc* m = reinterpret_cast<ChunkMisc*>(smem + Cfg::OFF_MISC);
    volatile int* abort = &m->abort;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = cluster_ctarank();
    int np = (int)(gridDim.x >> 1);
    const int pair = (int)(blockIdx.x >> 1);

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::NSLOT; ++i) {
            mbar_init(&m->full[i], 2);      // one arrival per CTA, with that CTA's bytes
            mbar_init(&m->empty[i], 1);
            mbar_init(&m->land[i], 1);
        }
        mbar_init(&m->q_full, 2);
        mbar_init(&m->q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&m->s_full[i], 1);
            mbar_init(&m->s_empty[i], 8);   // one arrival per softmax warp of both CTAs
            mbar_init(&m->p_full[i], 8);
            mbar_init(&m->p_empty[i], 1);
        }
        mbar_init(&m->o_full, 1);
        mbar_init(&m->o_empty, 8);
        mbar_init(&m->drain, 1);
        for (int i = 0; i < Cfg::NSEG; ++i) {
            mbar_init(&m->seg_full[i], 1);
            mbar_init(&m->seg_empty[i], crank == 0 ? 7 : 6);   // softmax, load and fixer warps; CTA 0: the issuer too
        }
        m->abort = 0;
        m->start_b = -1;
        fence_mbar_init();
    }
    if (warp == Cfg::MMA_WARP) {
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
    {
        int64_t mine = 0, excl;
        bool ok = true, all_ok = true;
        for (int b = threadIdx.x; b < p.B; b += Cfg::THREADS) {
            mine += chunk_seq(p, b, ok).blocks;
            all_ok = all_ok && ok;
        }
        if (!all_ok) atomicCAS(p.status, 0u, (uint32_t)kStBounds);
        total = block_scan(mine, m->sums, excl);
        // with fewer blocks than pairs, one each (the pairs behind them stay idle)
        np = (int)(total < np ? total : np);
        g0 = pair < np ? pair_start(total, pair, np) : 0;
        g1 = pair < np ? pair_start(total, pair + 1, np) : 0;
        int64_t base = 0;
        for (int b0 = 0; b0 < p.B && base <= g0 && g0 < g1; b0 += Cfg::THREADS) {
            const int b = b0 + (int)threadIdx.x;
            const int64_t v = b < p.B ? chunk_seq(p, b, ok).blocks : 0;
            const int64_t sum = block_scan(v, m->sums, excl);
            excl += base;
            if (v > 0 && excl <= g0 && g0 < excl + v) {
                m->start_b = b;
                m->start_before = excl;
            }
            base += sum;
        }
        __syncthreads();
    }

    if (warp == Cfg::SEG_WARP) {
        // ---------------------------------------------------------------- segments, loads of Q
        // The first tile by a search over 32 tiles at a time, the rest one by one.
        int b = m->start_b;
        int64_t g = g0;
        int tile = 0;
        int64_t tile_g0 = 0;               // the tile's first block in the list
        ChunkSeq s;
        bool sok;
        if (g0 < g1) {
            s = chunk_seq(p, b, sok);
            const int64_t want = g0 - m->start_before;
            int lo = 0, hi = s.tiles;      // the tile is in [lo, hi)
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32;
                const int i = lo + lane * step;
                const bool at = i < hi && tile_prefix(s, p.H, i) <= want;   // true for a prefix of the lanes
                const int nl = __popc(__ballot_sync(0xffffffffu, at));
                const int nlo = lo + (nl - 1) * step;
                hi = nlo + step < hi ? nlo + step : hi;
                lo = nlo;
            }
            tile = lo;
            tile_g0 = m->start_before + tile_prefix(s, p.H, tile);
        }
        // for the merge: first row, rows and pairs of the tile that starts here and ends in a later pair
        int4 head = make_int4(0, 0, 0, 0);
        bool ok = true;
        int ns = 0;
        if (lane == 0) {
            const uint32_t q_full = mapa_shared(smem_u32(&m->q_full), 0);
            while (true) {
                const int r = ns % Cfg::NSEG;
                if (!mbar_wait(&m->seg_empty[r], ((ns / Cfg::NSEG) & 1) ^ 1, abort, wlim)) {
                    ok = false;
                    break;
                }
                ChunkSeg sg;
                if (g >= g1) {
                    sg.b = -1;
                    m->seg[r] = sg;
                    mbar_arrive(&m->seg_full[r]);
                    break;
                }
                const int64_t nb = tile + 1 < s.tiles
                                       ? (tile + 1 + s.first) / p.H + 1
                                       : last_tile_blocks(s);
                const int r0 = tile * Cfg::ROWS;
                const int rows = s.rows - r0 < Cfg::ROWS ? s.rows - r0 : Cfg::ROWS;
                const int64_t stop = tile_g0 + nb < g1 ? tile_g0 + nb : g1;
                sg.b = b;
                sg.row0 = s.row0 + r0;
                sg.nrows = rows;
                sg.tok = r0 / p.H;
                sg.head = r0 % p.H;
                sg.c = s.c;
                sg.k0 = (int)(g - tile_g0);
                sg.k1 = (int)(stop - tile_g0);
                sg.see_all = s.c + sg.tok + 1;
                sg.see = s.c + (r0 + rows - 1) / p.H + 1;
                sg.part = sg.k0 == 0 && stop == tile_g0 + nb ? 0 : sg.k0 == 0 ? 1 : 2;
                sg.pad = 0;
                m->seg[r] = sg;
                mbar_arrive(&m->seg_full[r]);
                if (sg.part == 1)
                    head = make_int4(sg.row0, sg.nrows, pair_of_block(total, tile_g0 + nb - 1, np) - pair + 1, 0);
                // Q, once every QK of the segment before has completed
                if (ns > 0 && !mbar_wait(&m->q_empty, (ns - 1) & 1, abort, wlim)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx_cluster(q_full, Cfg::Q_BYTES);
                for (int kb = 0; kb < Cfg::KCH; ++kb)
                    tma_load_2d_pair(s_q + kb * 8192, &tm_q, q_full, kb * 64, sg.row0 + 64 * (int)crank);
                ++ns;
                g = stop;
                if (g < g1) {
                    // the next tile, of this sequence or of a later one
                    if (++tile == s.tiles) {
                        tile = 0;
                        do s = chunk_seq(p, ++b, sok);
                        while (s.blocks == 0 && b + 1 < p.B);
                    }
                    tile_g0 = g;
                }
            }
            if (!ok) *abort = 1;
            if (crank == 0) reinterpret_cast<int4*>(p.part)[pair] = head;
        }
        __syncwarp();
    } else if (warp == Cfg::LOAD_WARP) {
        // ---------------------------------------------------------------- loads of keys and values
        // test hook: the second CTA never loads
        bool ok = !(crank == 1 && (m->inject & 4u));
        uint32_t n = 0;                    // slots so far
        ChunkSeg sg = {};
        int pbase = 0, pid = -1;           // the lane's page id: page pbase + lane of the sequence
        auto refill = [&](int k) {
            pbase = 2 * k;
            const int page = pbase + lane;
            pid = -1;
            if (page < p.max_blocks && page * kPage < sg.see) {
                const int id = __ldg(p.block_table + (int64_t)sg.b * p.max_blocks + page);
                if (id >= 0 && id < p.num_blocks) pid = p.staged ? sg.b * p.staged + page : id;
                else atomicCAS(p.status, 0u, (uint32_t)kStBounds);
            }
        };
        auto slot_free = [&]() -> bool {
            const int r = n % Cfg::NSLOT;
            return __all_sync(0xffffffffu, mbar_wait(&m->empty[r], ((n / Cfg::NSLOT) & 1) ^ 1, abort, wlim));
        };
        auto load_keys = [&](int k) -> bool {
            const int id = __shfl_sync(0xffffffffu, pid, 2 * k + (int)crank - pbase);
            for (int kb = 0; kb < Cfg::KCH; ++kb) {
                if (!slot_free()) return false;
                const int r = n % Cfg::NSLOT;
                if (lane == 0) {
                    const uint32_t bar = mapa_shared(smem_u32(&m->full[r]), 0);
                    // a page that nobody sees is not loaded: its scores are replaced whatever they are
                    if (id >= 0) {
                        mbar_arrive_expect_tx_cluster(bar, Cfg::SLOT);
                        tma_load_2d_pair(s_ring + r * Cfg::SLOT, &tm_k, bar, kb * 64, id * kPage);
                    } else {
                        mbar_arrive_remote(bar);
                    }
                }
                __syncwarp();
                ++n;
            }
            return true;
        };
        auto load_values = [&](int k) -> bool {
            const ChunkBlock cb = chunk_block(sg, k);
            for (int g = 0; g < cb.ngroups; ++g) {
                const int id = __shfl_sync(0xffffffffu, pid, 2 * k + (g >> 1) - pbase);
                for (int h = 0; h < 2; ++h) {
                    if (!slot_free()) return false;
                    const int r = n % Cfg::NSLOT;
                    uint8_t* dst = s_ring + r * Cfg::SLOT;
                    const bool fix = g >= cb.fix_from;
                    if (id < 0) {          // a bad page id (reported): zeros
                        for (int i = lane; i < Cfg::SLOT / 16; i += 32)
                            reinterpret_cast<uint4*>(dst)[i] = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0) {
                        const uint32_t bar = mapa_shared(smem_u32(fix ? &m->land[r] : &m->full[r]), fix ? crank : 0);
                        if (id >= 0) {
                            const int x = 256 * h + 128 * (int)crank, y = id * kPage + 32 * (g & 1);
                            mbar_arrive_expect_tx_cluster(bar, Cfg::SLOT);
                            tma_load_2d_pair(dst, &tm_v, bar, x, y);
                            tma_load_2d_pair(dst + Cfg::SLOT / 2, &tm_v, bar, x + 64, y);
                        } else {
                            mbar_arrive_remote(bar);
                        }
                    }
                    __syncwarp();
                    ++n;
                }
            }
            return true;
        };
        for (int ns = 0; ok; ++ns) {
            const int r = ns % Cfg::NSEG;
            if (!__all_sync(0xffffffffu, mbar_wait(&m->seg_full[r], (ns / Cfg::NSEG) & 1, abort, wlim))) {
                ok = false;
                break;
            }
            sg = m->seg[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->seg_empty[r]);
            if (sg.b < 0) break;
            refill(sg.k0);
            ok = load_keys(sg.k0);
            for (int k = sg.k0; ok && k < sg.k1; ++k) {
                if (2 * (k + 1) + 1 >= pbase + 32) refill(k);
                if (k + 1 < sg.k1) ok = load_keys(k + 1);
                if (ok) ok = load_values(k);
            }
        }
        if (!ok) *abort = 1;
    } else if (warp == Cfg::FIX_WARP) {
        // ---------------------------------------------------------------- value rows at the causal edge
        bool ok = true;
        uint32_t n = 0, phase = 0;         // slots so far; next phase of each land barrier
        for (int ns = 0; ok; ++ns) {
            const int r = ns % Cfg::NSEG;
            if (!__all_sync(0xffffffffu, mbar_wait(&m->seg_full[r], (ns / Cfg::NSEG) & 1, abort, wlim))) {
                ok = false;
                break;
            }
            const ChunkSeg sg = m->seg[r];
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->seg_empty[r]);
            if (sg.b < 0) break;
            n += Cfg::KCH;                 // keys of the first block
            for (int k = sg.k0; ok && k < sg.k1; ++k) {
                if (k + 1 < sg.k1) n += Cfg::KCH;
                const ChunkBlock cb = chunk_block(sg, k);
                n += 2 * cb.fix_from;
                for (int g = cb.fix_from; ok && g < cb.ngroups; ++g)
                    for (int h = 0; ok && h < 2; ++h, ++n) {
                        const int sl = n % Cfg::NSLOT;
                        ok = __all_sync(0xffffffffu, mbar_wait(&m->land[sl], (phase >> sl) & 1, abort, wlim));
                        if (!ok) break;
                        phase ^= 1u << sl;
                        // lane = row of the group; its sixteen 16-byte pieces, in an order that
                        // spreads the lanes over the banks
                        uint8_t* row = s_ring + sl * Cfg::SLOT + lane * 128;
                        const int pos = k * Cfg::BLOCK + 32 * g + lane;
                        bool zero = pos >= sg.see;
                        if (!zero && pos >= sg.see_all) {
                            uint32_t bad = 0;
#pragma unroll
                            for (int q = 0; q < 16; ++q) {
                                const uint4 v = *reinterpret_cast<const uint4*>(
                                    row + (q >> 3) * (Cfg::SLOT / 2) + (((q + lane) & 7) << 4));
                                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    bad |= (uint32_t)((w[e] & 0x7F80u) == 0x7F80u) | (uint32_t)((w[e] & 0x7F800000u) == 0x7F800000u);
                            }
                            zero = bad != 0;
                        }
                        if (zero)
#pragma unroll
                            for (int q = 0; q < 16; ++q)
                                *reinterpret_cast<uint4*>(row + (q >> 3) * (Cfg::SLOT / 2) + (((q + lane) & 7) << 4)) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) arrive_leader(&m->full[sl], crank);
                    }
            }
        }
        if (!ok) *abort = 1;
    } else if (warp == Cfg::MMA_WARP) {
        if (crank == 0) {
            // ------------------------------------------------------------ MMA issuer
            bool ok = true;
            if (lane == 0) {
                const uint32_t q_addr = smem_u32(s_q), p_addr = smem_u32(s_p), r_addr = smem_u32(s_ring);
                uint32_t n = 0, blk = 0;   // slots and blocks so far
                auto slot = [&](uint32_t& addr) -> bool {
                    const int r = n % Cfg::NSLOT;
                    addr = r_addr + r * Cfg::SLOT;
                    if (!mbar_wait(&m->full[r], (n / Cfg::NSLOT) & 1, abort, wlim)) return false;
                    tc_fence_after();
                    return true;
                };
                auto issue_qk = [&](uint32_t bi, bool last) -> bool {
                    const int b = bi & 1;
                    if (!mbar_wait(&m->s_empty[b], ((bi >> 1) & 1) ^ 1, abort, wlim)) return false;
                    tc_fence_after();
                    for (int kb = 0; kb < Cfg::KCH; ++kb) {
                        uint32_t a;
                        if (!slot(a)) return false;
#pragma unroll
                        for (int k16 = 0; k16 < 4; ++k16)
                            umma_bf16_2cta(tm_s + b * 64, sdesc_sw128(q_addr + kb * 8192 + k16 * 32, 16, 1024),
                                           sdesc_sw128(a + k16 * 32, 16, 1024), Cfg::IDESC_QK, (kb | k16) != 0);
                        umma_commit_2cta(&m->empty[n % Cfg::NSLOT], 3);
                        ++n;
                    }
                    umma_commit_2cta(&m->s_full[b], 3);
                    if (last) umma_commit_2cta(&m->q_empty, 3);
                    return true;
                };
                auto issue_pv = [&](uint32_t bi, const ChunkBlock& cb, bool first, bool last, int ns) -> bool {
                    const int b = bi & 1;
                    if (!mbar_wait(&m->p_full[b], (bi >> 1) & 1, abort, wlim)) return false;
                    // O of the segment before must have been read by both epilogues
                    if (first && ns > 0 && !mbar_wait(&m->o_empty, (ns - 1) & 1, abort, wlim)) return false;
                    tc_fence_after();
                    for (int g = 0; g < cb.ngroups; ++g)
                        for (int h = 0; h < 2; ++h) {
                            uint32_t a;
                            if (!slot(a)) return false;
#pragma unroll
                            for (int s16 = 0; s16 < 2; ++s16)
                                // A = P [64 rows x 16 positions] K-major; B = V [16 positions x 128
                                // columns per CTA] MN-major: 64-column chunks half a slot apart (LBO),
                                // 8-row groups 1024 B (SBO)
                                umma_bf16_2cta(tm_o + h * 128,
                                               sdesc_sw128(p_addr + b * Cfg::P_BYTES + (g >> 1) * 8192 +
                                                               ((g & 1) * 2 + s16) * 32, 16, 1024),
                                               sdesc_sw128(a + s16 * 16 * 128, Cfg::SLOT / 2, 1024), Cfg::IDESC_PV,
                                               !first || g > 0 || s16 > 0);
                            umma_commit_2cta(&m->empty[n % Cfg::NSLOT], 3);
                            ++n;
                        }
                    umma_commit_2cta(&m->p_empty[b], 3);
                    if (last) umma_commit_2cta(&m->o_full, 3);
                    return true;
                };
                for (int ns = 0; ok; ++ns) {
                    const int r = ns % Cfg::NSEG;
                    if (!mbar_wait(&m->seg_full[r], (ns / Cfg::NSEG) & 1, abort, wlim)) {
                        ok = false;
                        break;
                    }
                    const ChunkSeg sg = m->seg[r];
                    mbar_arrive(&m->seg_empty[r]);
                    if (sg.b < 0) break;
                    ok = mbar_wait(&m->q_full, ns & 1, abort, wlim);
                    if (!ok) break;
                    tc_fence_after();
                    ok = issue_qk(blk, sg.k0 + 1 == sg.k1);
                    for (int k = sg.k0; ok && k < sg.k1; ++k, ++blk) {
                        if (k + 1 < sg.k1) ok = issue_qk(blk + 1, k + 2 == sg.k1);
                        if (ok) ok = issue_pv(blk, chunk_block(sg, k), k == sg.k0, k + 1 == sg.k1, ns);
                    }
                }
                volatile int no_abort = 0;
                umma_commit_2cta(&m->drain, 1);
                mbar_wait(&m->drain, 0, &no_abort, wlim);
                if (!ok) *abort = 1;
            }
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------- softmax + epilogue
        const int L = threadIdx.x;                   // TMEM lane
        const int hl = L & 63;                       // row of this CTA's 64
        const int half = L >> 6;                     // positions 64*half.. of a block; value columns of this half
        const int rr = 64 * (int)crank + hl;         // row of the tile
        const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
        auto col_of = [&](int c0) { return c0 < 128 ? 128 * half + c0 : 256 + 128 * half + (c0 - 128); };
        uint32_t blk = 0;
        bool ok = true;
        // Every exit decision of these 128 threads is taken together (votes carried
        // by named barriers), so the named barriers always match.
        for (int ns = 0;; ++ns) {
            const int sr = ns % Cfg::NSEG;
            const bool there = mbar_wait(&m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim);
            ok = named_bar_and(1, 128, ok && there);
            if (!ok) break;
            const ChunkSeg sg = m->seg[sr];
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
            bool next_ok = page_ok(sg.k0);
            float mrun = -INFINITY, lrun = 0.0f, lfull = 0.0f;
            for (int k = sg.k0; k < sg.k1; ++k, ++blk) {
                const int b = blk & 1;
                const uint32_t u = (blk >> 1) & 1;
                const bool this_ok = next_ok;
                if (k + 1 < sg.k1) next_ok = page_ok(k + 1);
                const bool got = __all_sync(0xffffffffu, mbar_wait(&m->s_full[b], u, abort, wlim));
                float sv[64];
                float mx = -INFINITY;
                if (got) {
                    tc_fence_after();
                    uint32_t a[32], a2[32];
                    tmem_ld32(tm_s + lane_off + b * 64, a);
                    tmem_ld32(tm_s + lane_off + b * 64 + 32, a2);
                    tmem_wait_ld();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) arrive_leader(&m->s_empty[b], crank);
                    int vis = see - (k * Cfg::BLOCK + 64 * half);     // positions of this half that the row sees
                    if (!this_ok) vis = 0;
                    if (__all_sync(0xffffffffu, vis >= 64)) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            sv[i] = __uint_as_float(a[i]) * p.scale_log2;
                            sv[32 + i] = __uint_as_float(a2[i]) * p.scale_log2;
                            mx = fmaxf(mx, fmaxf(sv[i], sv[32 + i]));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            sv[i] = i < vis ? __uint_as_float(a[i]) * p.scale_log2 : -INFINITY;
                            sv[32 + i] = 32 + i < vis ? __uint_as_float(a2[i]) * p.scale_log2 : -INFINITY;
                            mx = fmaxf(mx, fmaxf(sv[i], sv[32 + i]));
                        }
                    }
                }
                // the row's other 64 positions are in lane L^64 (two exchange buffers, so the next
                // block's write cannot meet this read)
                float* xm = s_xm + b * 128;
                xm[L] = mx;
                ok = named_bar_and(1, 128, ok && got);
                if (!ok) break;
                const float mnew = fmaxf(mrun, fmaxf(mx, xm[L ^ 64]));
                const bool rescale = mnew > mrun + 8.0f;      // identical in both lanes of a row
                const float muse = rescale ? mnew : mrun;
                const bool none = muse == -INFINITY;
                uint32_t pk[32];
                float r0 = 0.0f, r1 = 0.0f, f0 = 0.0f, f1 = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float p0 = none ? 0.0f : fast_exp2(sv[2 * i] - muse);
                    const float p1 = none ? 0.0f : fast_exp2(sv[2 * i + 1] - muse);
                    pk[i] = pack_bf16(p0, p1);
                    // O is divided by the sum of the bf16 weights that the MMA multiplies (their
                    // roundings cancel in part); lse takes the sum before rounding
                    r0 += __uint_as_float(pk[i] << 16);
                    r1 += __uint_as_float(pk[i] & 0xFFFF0000u);
                    f0 += p0;
                    f1 += p1;
                }
                // P buffer b is free once P.V of block blk-2 completed
                ok = __all_sync(0xffffffffu, mbar_wait(&m->p_empty[b], u ^ 1, abort, wlim));
                const bool need = rescale && k > sg.k0;
                float f = 1.0f;
                if (need) f = fast_exp2(mrun - muse);
                if (ok && __any_sync(0xffffffffu, need)) {
                    // O must be stable: P.V of the block before has completed.  TMEM loads and
                    // stores are warp-wide: lanes whose row keeps its max scale by 1.
                    ok = __all_sync(0xffffffffu, mbar_wait(&m->p_empty[b ^ 1], ((blk - 1) >> 1) & 1, abort, wlim));
                    if (ok) {
                        tc_fence_after();
#pragma unroll 1
                        for (int c0 = 0; c0 < 256; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(tm_o + lane_off + c0, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                            tmem_st32(tm_o + lane_off + c0, o);
                        }
                        tmem_wait_st();
                    }
                }
                lrun = lrun * f + (r0 + r1);
                lfull = lfull * f + (f0 + f1);
                mrun = muse;
                if (ok) {
                    // P row hl, chunk of this half: eight 16-byte pieces of a 128-byte row (128-byte swizzle)
                    uint8_t* prow = s_p + b * Cfg::P_BYTES + half * 8192 + hl * 128;
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<uint4*>(prow + ((((uint32_t)q) ^ (uint32_t)(hl & 7)) << 4)) =
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
            // the row's sums: this lane's positions plus the partner lane's
            const bool ofull = ok && mbar_wait(&m->o_full, ns & 1, abort, wlim);
            if (!named_bar_and(1, 128, ofull)) {
                ok = false;
                break;
            }
            s_xm[L] = lrun;
            s_xm[128 + L] = lfull;
            named_bar_sync(1, 128);
            const float ltot = lrun + s_xm[L ^ 64];
            const float lft = lfull + s_xm[128 + (L ^ 64)];
            tc_fence_after();
            const bool empty = ltot == 0.0f;   // the row saw nothing here
            const int64_t row = (int64_t)sg.row0 + rr;
            if (sg.part == 0) {
                const float inv = empty ? 0.0f : 1.0f / ltot;
                for (int c0 = 0; c0 < 256; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tm_o + lane_off + c0, o);
                    tmem_wait_ld();
                    if (real) {
                        uint4* dst = reinterpret_cast<uint4*>(p.out + row * kDv + col_of(c0));
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = empty ? 0.0f : __uint_as_float(o[i + e]) * inv;
                            dst[i / 8] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                                    pack_bf16(v[6], v[7]));
                        }
                    }
                }
                if (half == 0 && real && p.lse)
                    p.lse[row] = empty ? -INFINITY : (mrun + log2f(lft)) * 0.69314718055994531f;
            } else {
                uint8_t* sl = p.part + Cfg::HEAD_BYTES +
                              ((int64_t)(2 * pair + (sg.part == 1 ? 1 : 0)) * 2 + crank) * Cfg::PART_BYTES;
                float* od = reinterpret_cast<float*>(sl) + hl * 512;
                for (int c0 = 0; c0 < 256; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld32(tm_o + lane_off + c0, o);
                    tmem_wait_ld();
                    if (real)
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            __stcg(reinterpret_cast<uint4*>(od + col_of(c0) + i),
                                   empty ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]));
                }
                if (half == 0 && real)
                    __stcg(reinterpret_cast<float4*>(sl + Cfg::PART_O) + hl,
                           make_float4(empty ? -INFINITY : mrun, ltot, lft, 0.0f));
            }
            // O has been read: the next segment's first P.V may overwrite it
            tc_fence_before();
            named_bar_sync(1, 128);
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
    if (warp == Cfg::MMA_WARP) {
        tc_fence_after();
        tmem_dealloc_2cta(tmem_base, Cfg::TMEM_COLS);
    }
    if (threadIdx.x == 0 && m->abort) atomicCAS(p.status, 0u, (uint32_t)kStTimeout);
}

// Merge of the tiles whose blocks were spread over several pairs.  Block (x, y):
// rows 8y.. of the tile that starts in pair x and ends in a later one (none: no
// splits), one warp per row.  Split s of the tile is pair x + s's; with m_s its
// running maximum (log2 units), l_s and e_s its sums of weights,
//   O = sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s,
//   lse = (M + log2 sum_s 2^(m_s - M) e_s) ln 2,  M = max m_s,
// added up in split order.
__global__ void __launch_bounds__(ChunkCfg::COMBINE_THREADS) chunk_combine_kernel(const __grid_constant__ ChunkParams p) {
    using Cfg = ChunkCfg;
    griddep_wait();
    const int pair = (int)blockIdx.x;
    const int row = (int)blockIdx.y * (Cfg::COMBINE_THREADS / 32) + (int)(threadIdx.x >> 5);
    const int lane = (int)(threadIdx.x & 31);
    const int4 head = __ldcg(reinterpret_cast<const int4*>(p.part) + pair);
    const int S = head.z;
    if (row >= head.y || S < 2) return;
    const int crank = row >> 6, hl = row & 63;
    auto slot = [&](int s) -> const uint8_t* {
        return p.part + Cfg::HEAD_BYTES + ((int64_t)(2 * (pair + s) + (s == 0 ? 1 : 0)) * 2 + crank) * Cfg::PART_BYTES;
    };
    constexpr int PER = Cfg::MAX_PAIRS / 32;
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
    float4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < PER; ++j)
        for (int i = 0; i < 32 && 32 * j + i < S; ++i) {
            const float ws = __shfl_sync(0xffffffffu, w[j], i);
            if (ws == 0.0f) continue;
            const float4* o = reinterpret_cast<const float4*>(slot(32 * j + i)) + hl * 128 + lane;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 v = __ldcg(o + 32 * q);
                acc[q].x = fmaf(ws, v.x, acc[q].x);
                acc[q].y = fmaf(ws, v.y, acc[q].y);
                acc[q].z = fmaf(ws, v.z, acc[q].z);
                acc[q].w = fmaf(ws, v.w, acc[q].w);
            }
        }
    const bool empty = l == 0.0f;
    const float inv = empty ? 0.0f : 1.0f / l;
    uint2* dst = reinterpret_cast<uint2*>(p.out + ((int64_t)head.x + row) * kDv) + lane;
#pragma unroll
    for (int q = 0; q < 4; ++q)
        dst[32 * q] = make_uint2(pack_bf16(acc[q].x * inv, acc[q].y * inv), pack_bf16(acc[q].z * inv, acc[q].w * inv));
    if (lane == 0 && p.lse) p.lse[(int64_t)head.x + row] = empty ? -INFINITY : (M + log2f(e)) * 0.69314718055994531f;
}

// ------------------------------------------------------------------ FP8 latent cache
// The pages of every sequence, dequantized to bf16 (code x tile scale, rounded
// once) into a copy that is laid out by sequence: page i of sequence b at
// b * pages + i.  One block per page: its 64 rows are 2304 runs of 16 codes,
// nine per thread, all loaded before any is converted.  Memory-bound: reads 596
// bytes a row and writes 1152.
struct PagesParams {
    const int32_t* seq_lens;
    const int32_t* block_table;
    const uint8_t* codes;       // [num_blocks * 64, 576]
    const float* scale;         // [num_blocks * 64, 5]
    uint16_t* rows;             // [B * pages * 64, 576] bf16 bits
    int32_t B, max_blocks, num_blocks, pages;
};

constexpr int kPagesThreads = 256;

__global__ void __launch_bounds__(kPagesThreads) kv_fp8_pages_kernel(const __grid_constant__ PagesParams p) {
    griddep_launch_dependents();
    const int b = (int)blockIdx.x / p.pages, page = (int)blockIdx.x % p.pages;
    if ((int64_t)page * kPage >= __ldg(p.seq_lens + b) || page >= p.max_blocks) return;
    const int id = __ldg(p.block_table + (int64_t)b * p.max_blocks + page);
    if (id < 0 || id >= p.num_blocks) return;          // the attention kernel reports it and does not read the copy
    constexpr int RUNS = kPage * kDqk / 16, PER = RUNS / kPagesThreads;
    static_assert(RUNS % kPagesThreads == 0, "whole runs per thread");
    const uint4* src = reinterpret_cast<const uint4*>(p.codes + (int64_t)id * kPage * kDqk);
    const float* sc = p.scale + (int64_t)id * kPage * kKvTiles;
    uint4* dst = reinterpret_cast<uint4*>(p.rows + ((int64_t)b * p.pages + page) * kPage * kDqk);
    uint4 v[PER];
    float s[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = i * kPagesThreads + (int)threadIdx.x;
        v[i] = __ldg(src + r);
        s[i] = __ldg(sc + r / 36 * kKvTiles + r % 36 / 8);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int r = i * kPagesThreads + (int)threadIdx.x;
        stage_chunk(v[i], s[i], dst + 2 * r);
    }
}

}  // namespace dsa
