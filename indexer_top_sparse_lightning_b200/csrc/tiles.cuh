// tiles.cuh -- the work list of the kernels that run new tokens densely against
// the paged cache, and waits shared by their roles.
//
// The (token, head) rows of a sequence's new tokens, token-major, are cut into
// tiles of ROWS rows, and the positions that a tile sees into blocks of BLOCK.
// All blocks of all tiles form one list, of which every pair of CTAs takes an
// even, contiguous share.  The list is never stored: the blocks of a sequence's
// first i tiles have a closed form.
#pragma once
#include "common.h"
#include "pair.cuh"
#include "ptx.cuh"

namespace dsa {

// What the list is made of.
struct ListParams {
    const int32_t* seq_lens;
    const int32_t* cu_q;
    const int32_t* block_table;
    int32_t B, T, H, max_blocks, num_blocks;
    int32_t staged;           // > 0: the cache is an fp16 copy by sequence, `staged` pages each
    int32_t max_len;          // longest cached length that the buffers have room for
    int32_t tok0, tokens;     // the new tokens tok0 .. tok0 + tokens - 1 of each sequence
    int32_t max_tokens;       // most new tokens of a sequence that the launches cover
};

// One sequence as the list sees it.
struct ChunkSeq {
    int32_t row0, rows;       // its (token, head) rows, over the whole batch
    int32_t c, n, len;        // position of its first token here, tokens here, cached length
    int32_t tiles, first;     // tiles; (c * H - 1) / ROWS, rounded down
    int64_t blocks;           // blocks of all tiles
};

// A run of blocks of one tile.
struct TileRun {
    int32_t b;                // sequence, -1: no more runs
    int32_t tile;             // in its sequence
    int32_t row0;             // first (token, head) row of the tile, over the whole batch
    int32_t nrows;            // rows of the tile (up to ROWS)
    int32_t tok, head;        // token (counted like c) and head of that row
    int32_t c;                // position of token 0
    int32_t k0, k1;           // blocks
    int32_t see_all, see;     // positions below see_all are seen by every row, none at or above see by any
    int32_t part;             // 0: the whole tile; 1: its first blocks; 2: later blocks
};

// Where a pair's share starts.
struct ShareStart {
    ChunkSeq seq;
    int64_t before;           // blocks before that sequence
    int32_t b;
    int32_t pad;
};

// sum over x < n of floor(x / h)
__device__ __forceinline__ int64_t floor_sum(uint32_t n, uint32_t h) {
    const uint32_t q = n / h, r = n % h;
    return (int64_t)h * q * (q > 0 ? q - 1 : 0) / 2 + (int64_t)r * q;
}

// pair_start and pair_of_block, without 64-bit divisions for lists of ordinary length.
__device__ __forceinline__ int64_t share_start(int64_t total, int pr, int np) {
    return total < (1 << 24) ? (int64_t)((uint32_t)total * (uint32_t)pr / (uint32_t)np) : pair_start(total, pr, np);
}
__device__ __forceinline__ int share_of(int64_t total, int64_t g, int np) {
    return total < (1 << 24) ? (int)(((uint32_t)(g + 1) * (uint32_t)np + (uint32_t)total - 1) / (uint32_t)total) - 1
                             : pair_of_block(total, g, np);
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

template <int ROWS, int BLOCK>
struct TileList {
    static_assert(BLOCK % ROWS == 0, "the closed form needs whole tiles per block of one head");
    static constexpr int G = BLOCK / ROWS;

    // Blocks of the tiles before tile i (i < tiles).  Tile k < tiles - 1 ends with row
    // ROWS (k + 1) - 1, so it sees c + floor((ROWS (k + 1) - 1) / H) + 1 positions, in
    // floor((c + floor((ROWS (k + 1) - 1) / H)) / BLOCK) + 1 blocks, which is
    // floor((k + 1 + first) / (G H)) + 1 with first = floor((c H - 1) / ROWS) (nested
    // floors of quotients by integers commute).
    static __device__ __forceinline__ int64_t prefix(const ChunkSeq& s, int H, int i) {
        return (int64_t)i + floor_sum((uint32_t)(i + 1 + s.first), (uint32_t)(G * H)) -
               floor_sum((uint32_t)(1 + s.first), (uint32_t)(G * H));
    }
    static __device__ __forceinline__ int64_t blocks(const ChunkSeq& s, int H, int i) {
        return (i + 1 < s.tiles ? (i + 1 + s.first) / (G * H) : (s.c + s.n - 1) / BLOCK) + 1;
    }

    // Sequence b, with sizes that no input can push out of range: a length is cut to max_len, tokens in
    // front of position 0 (a length below their number) and tokens past T are left out, all reported by
    // `ok`.  Token j of nq stands at len - nq + j whatever is left out.
    static __device__ __forceinline__ ChunkSeq seq(const ListParams& p, int b, bool& ok) {
        ChunkSeq s;
        const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), len = __ldg(p.seq_lens + b);
        const int64_t nq = q1 > q0 ? (int64_t)q1 - q0 : 0;
        ok = q0 >= 0 && q1 >= q0 && q1 <= p.T && len <= p.max_len && (q1 == q0 || len >= nq) && nq <= p.max_tokens;
        s.len = len < 0 ? 0 : len > p.max_len ? p.max_len : len;
        const int64_t first = (int64_t)q1 - (nq < s.len ? nq : s.len);      // the token at position 0 or the first one
        const int lo = first < 0 ? 0 : first > p.T ? p.T : (int)first, hi = q1 < lo ? lo : q1 > p.T ? p.T : q1;
        const int n = hi - lo;
        s.c = s.len - (int)(q1 - (int64_t)lo) + p.tok0;
        s.n = n - p.tok0 < p.tokens ? n - p.tok0 : p.tokens;
        if (s.n < 0) s.n = 0;
        s.row0 = (lo + p.tok0) * p.H;
        s.rows = s.n * p.H;
        s.tiles = (s.rows + ROWS - 1) / ROWS;
        const int64_t ch = (int64_t)s.c * p.H;
        s.first = ch > 0 ? (int)((ch - 1) / ROWS) : -1;
        s.blocks = s.tiles > 0 ? prefix(s, p.H, s.tiles - 1) + blocks(s, p.H, s.tiles - 1) : 0;
        return s;
    }

    // The share [g0, g1) of this pair, and where it starts (by all THREADS threads of the block).
    // `np` is cut to the length of the list: with fewer blocks than pairs, one each (the pairs
    // behind them stay idle).
    template <int THREADS>
    static __device__ __forceinline__ void share(const ListParams& p, int pair, int& np, int64_t* sums, ShareStart* start,
                                                 uint32_t* status, int64_t& g0, int64_t& g1, int64_t& total) {
        // the first THREADS sequences stay with their threads; more are counted, and looked for, in turns
        int64_t excl;
        bool ok = true, all_ok = true;
        const ChunkSeq own = (int)threadIdx.x < p.B ? seq(p, (int)threadIdx.x, all_ok) : ChunkSeq{};
        int64_t mine = 0;
        for (int b = (int)threadIdx.x + THREADS; b < p.B; b += THREADS) {
            mine += seq(p, b, ok).blocks;
            all_ok = all_ok && ok;
        }
        if (!all_ok) atomicCAS(status, 0u, (uint32_t)kStBounds);
        const int64_t first = block_scan(own.blocks, sums, excl);
        total = first;
        if (p.B > THREADS) {
            int64_t unused;
            total += block_scan(mine, sums, unused);
        }
        np = (int)(total < np ? total : np);
        g0 = pair < np ? share_start(total, pair, np) : 0;
        g1 = pair < np ? share_start(total, pair + 1, np) : 0;
        auto claim = [&](int b, const ChunkSeq& q, int64_t before) {
            if (q.blocks > 0 && before <= g0 && g0 < before + q.blocks) {
                start->b = b;
                start->before = before;
                start->seq = q;
            }
        };
        claim((int)threadIdx.x, own, excl);
        int64_t base = first;
        for (int b0 = THREADS; b0 < p.B && base <= g0 && g0 < g1; b0 += THREADS) {
            const int b = b0 + (int)threadIdx.x;
            const ChunkSeq q = b < p.B ? seq(p, b, ok) : ChunkSeq{};
            const int64_t sum = block_scan(q.blocks, sums, excl);
            claim(b, q, base + excl);
            base += sum;
        }
        __syncthreads();
    }

    // The runs of a share, one after another (by one warp; `at` of all lanes).
    struct Walk {
        ChunkSeq s;
        int64_t g, g1, tile_g0;    // next block, end of the share, the tile's first block in the list
        int b, tile;
    };
    // The share's first tile, by a search over 32 tiles at a time.
    static __device__ __forceinline__ Walk begin(const ListParams& p, const ShareStart& start, int64_t g0, int64_t g1) {
        Walk w;
        w.g = g0;
        w.g1 = g1;
        w.b = 0;
        w.tile = 0;
        w.tile_g0 = 0;
        w.s = ChunkSeq{};
        if (g0 < g1) {
            const int lane = threadIdx.x & 31;
            w.b = start.b;
            w.s = start.seq;
            const int64_t want = g0 - start.before;
            int lo = 0, hi = w.s.tiles;    // the tile is in [lo, hi)
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32;
                const int i = lo + lane * step;
                const bool at = i < hi && prefix(w.s, p.H, i) <= want;   // true for a prefix of the lanes
                const int nl = __popc(__ballot_sync(0xffffffffu, at));
                const int nlo = lo + (nl - 1) * step;
                hi = nlo + step < hi ? nlo + step : hi;
                lo = nlo;
            }
            w.tile = lo;
            w.tile_g0 = start.before + prefix(w.s, p.H, lo);
        }
        return w;
    }
    // The run at w.g (w.g < w.g1); `nb` receives the blocks of its whole tile.
    static __device__ __forceinline__ TileRun run(const ListParams& p, const Walk& w, int64_t& nb) {
        TileRun r;
        nb = blocks(w.s, p.H, w.tile);
        const int r0 = w.tile * ROWS;
        const int64_t stop = w.tile_g0 + nb < w.g1 ? w.tile_g0 + nb : w.g1;
        r.b = w.b;
        r.tile = w.tile;
        r.row0 = w.s.row0 + r0;
        r.nrows = w.s.rows - r0 < ROWS ? w.s.rows - r0 : ROWS;
        r.tok = r0 / p.H;
        r.head = r0 % p.H;
        r.c = w.s.c;
        r.k0 = (int)(w.g - w.tile_g0);
        r.k1 = (int)(stop - w.tile_g0);
        r.see_all = w.s.c + r.tok + 1;
        r.see = w.s.c + (r0 + r.nrows - 1) / p.H + 1;
        r.part = r.k0 == 0 && r.k1 == nb ? 0 : r.k0 == 0 ? 1 : 2;
        return r;
    }
    // To the next run.
    static __device__ __forceinline__ void next(const ListParams& p, Walk& w, const TileRun& r) {
        w.g += r.k1 - r.k0;
        if (w.g >= w.g1) return;
        if (++w.tile == w.s.tiles) {
            bool ok;
            w.tile = 0;
            do w.s = seq(p, ++w.b, ok);
            while (w.s.blocks == 0 && w.b + 1 < p.B);
        }
        w.tile_g0 = w.g;
    }
};

// log2 of a power of two (a normal number).
__device__ __forceinline__ float log2_of_power(float f) { return (float)((int)(__float_as_uint(f) >> 23) - 127); }

// Waits of a whole warp: one lane polls (32 lanes' polls would each take a turn in
// the shared-memory pipe that every other barrier operation needs), the rest
// sleep at the warp's barrier.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    int ok = 1;
    if ((threadIdx.x & 31) == 0) ok = mbar_spin(bar, parity, abort, limit_ns);
    __syncwarp();
    return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// The same in warps that act through an elected lane; the answer is uniform.
__device__ __forceinline__ bool elected_wait(bool el, uint64_t* bar, uint32_t parity, volatile int* abort,
                                             uint64_t limit_ns) {
    bool ok = true;
    if (el) ok = mbar_spin(bar, parity, abort, limit_ns);
    return __all_sync(0xffffffffu, ok);
}

}  // namespace dsa
