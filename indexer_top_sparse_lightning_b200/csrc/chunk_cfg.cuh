// chunk_cfg.cuh -- layout, barriers and parameters of the dense attention kernel
// (chunk.cuh), shared with the roles that convert an FP8 cache (chunk_fp8.cuh).
#pragma once
#include "common.h"
#include "pair.cuh"
#include "ptx.cuh"
#include "tiles.cuh"

namespace dsa {

// Where keys and values come from: bf16 rows; e4m3 codes, converted in the kernel; the fp16
// copy of an FP8 cache.
enum ChunkCache { kCacheBf16, kCacheFp8, kCacheCopy };

struct ChunkCfg {
    static constexpr int ROWS = 128;                    // (token, head) rows of a tile
    static constexpr int BLOCK = 128;                   // positions of a block (two pages)
    static constexpr int KCH = 9;                       // 64-column chunks of a latent row
    static constexpr int KRING = 3;                     // groups of keys that are kept
    static constexpr int KGROUP = 3 * 8192;             // 64 rows x 3 chunks; three make a block, six over the fp16 copy
    static constexpr int VGROUPS = 4;                   // groups of a block's values: 32 rows x 4 chunks (this CTA's)
    static constexpr int VRING = 3;                     // groups that are kept
    static constexpr int VGROUP = 4 * 4096;
    // FP8: converted groups of keys (64 rows x 2 chunks, five make a block) and of values (32 rows
    // x 4 chunks), and groups of codes on their way there
    static constexpr int FGROUP = 16384;
    static constexpr int CGROUP = 8192;
    static constexpr int FKRING = 2, FVRING = 3;        // (three and two: 536 us for 524)
    static constexpr int TILES = 5;                     // scales of a position
    static constexpr int NREC = 3;                      // blocks whose position factors are kept
    static constexpr int CONV_WARPS = 4;                // warps that convert keys, and as many for values
    static constexpr int Q_BYTES = KCH * 64 * 128;      // this CTA's 64 rows
    static constexpr int P_BYTES = 64 * BLOCK * 2;      // [64 rows x 128 positions] bf16: two 64-position chunks
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_P = OFF_Q + Q_BYTES;
    static constexpr int OFF_K = OFF_P + 2 * P_BYTES;
    static constexpr int OFF_V = OFF_K + KRING * KGROUP;
    static constexpr int OFF_XM = OFF_V + VRING * VGROUP;   // exchange between the threads of a row
    // FP8: one weight buffer, keys, values, codes of keys and of values, position factors
    static constexpr int OFF_FK = OFF_P + P_BYTES;
    static constexpr int OFF_FV = OFF_FK + FKRING * FGROUP;
    static constexpr int OFF_KC = OFF_FV + FVRING * FGROUP;
    static constexpr int OFF_VC = OFF_KC + FKRING * CGROUP;
    static constexpr int OFF_REC = OFF_VC + FVRING * CGROUP;
    static constexpr int OFF_MISC = OFF_XM + 256 * 4;
    static constexpr int MISC_BYTES = 1024;
    static constexpr int SMEM = 1024 + OFF_MISC + MISC_BYTES;
    static constexpr int SOFTMAX_WARPS = 8;
    static constexpr int warps(bool fp8) { return fp8 ? 16 + 2 * CONV_WARPS : 14; }
    static constexpr int MAX_WARPS = 16 + 2 * CONV_WARPS;
    // A row's reference (a maximum minus DROP) is replaced once a score exceeds it by more than LAZY.
    // bf16 weights and fp32 sums are floating point, so a reference below the maximum costs no
    // precision, and 2^32 (2^52 for the sums of a million weights) is far from fp32's range; a
    // replacement waits for the P.V in flight.  fp16 weights end at 2^16 and lose bits below
    // 2^-14: references seven below the maximum keep them in [2^-14, 2^15] down to 2^-21 of the
    // largest weight, and to 2^-32 of it with an absolute error.
    static constexpr float lazy(bool fp16) { return fp16 ? 15.0f : 32.0f; }
    static constexpr float drop(bool fp16) { return fp16 ? 7.0f : 0.0f; }
    static constexpr int NSEG = 4;                      // segment ring
    static constexpr int TMEM_COLS = 512;               // O: [0, 256); from column 256 two score buffers of 64, or (FP8) one of 4 x 64
    // fp16 operands: the bf16 descriptor without its two operand-format bits
    static constexpr uint32_t BF16_BITS = (1u << 7) | (1u << 10);
    static constexpr uint32_t idesc_qk(bool fp16) { return idesc_bf16_f32(128, BLOCK, false, false) & ~(fp16 ? BF16_BITS : 0u); }
    static constexpr uint32_t idesc_pv(bool fp16) { return idesc_bf16_f32(128, 256, false, true) & ~(fp16 ? BF16_BITS : 0u); }
    // partial result of (pair, side, CTA): O [64 rows][512] fp32, then (m, sum, sum for lse, -) per row.
    // Side 1: the pair holds the tile's first blocks; side 0: later ones.
    static constexpr int64_t PART_O = 64 * 512 * 4;
    static constexpr int64_t PART_BYTES = PART_O + 64 * 16;
    static constexpr int64_t HEAD_BYTES = 2048;         // one int4 per pair: the tile that starts there and ends in a later pair
    static constexpr int MAX_PAIRS = 128;                // the merge keeps four splits per lane
    static constexpr int COMBINE_THREADS = 512;         // at least MAX_PAIRS
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
    const uint8_t* codes;     // FP8: [num_blocks * 64, 576] e4m3 codes, [num_blocks * 64, 5] scales
    const float* kv_scale;
    const float* page_scale;  // fp16 copy: the power-of-two factor of each page, [B, staged]
    float scale_log2;         // sm_scale * log2(e)
};

struct ChunkMisc {
    uint64_t k_full[ChunkCfg::KRING];   // (CTA 0) the key group is ready in both CTAs
    uint64_t k_empty[ChunkCfg::KRING];  // its MMAs have completed (FP8: and codes for it have landed)
    uint64_t v_full[ChunkCfg::VRING];   // (CTA 0) the value group is ready in both CTAs
    uint64_t v_empty[ChunkCfg::VRING];
    uint64_t v_peer[ChunkCfg::VRING];     // (CTA 0) CTA 1's fixer is done with the group
    uint64_t v_land[ChunkCfg::VRING];   // the group has landed, for the fixer to look at
    uint64_t q_full;                      // (CTA 0) Q of both CTAs
    uint64_t q_land;                      // (FP8) this CTA's Q, still bf16
    uint64_t rec_full[ChunkCfg::NREC], rec_empty[ChunkCfg::NREC];   // (FP8) position factors
    uint64_t kc_empty[ChunkCfg::FKRING], vc_empty[ChunkCfg::FVRING]; // (FP8) codes have been converted
    uint64_t q_empty;
    uint64_t s_full[2], s_empty[2];       // per score buffer; FP8: of accumulator 3, of the others
    uint64_t p_full[2], p_empty[2];
    uint64_t o_full, o_empty, drain[2];
    uint64_t seg_full[ChunkCfg::NSEG], seg_empty[ChunkCfg::NSEG];
    TileRun seg[ChunkCfg::NSEG];
    uint64_t wait_ns;
    ShareStart start;
    int64_t sums[ChunkCfg::MAX_WARPS];
    uint32_t tmem_base;
    int abort;
    uint32_t inject;
};
static_assert(sizeof(ChunkMisc) <= ChunkCfg::MISC_BYTES, "misc block exceeds its slot");

// FP8: the factors of a block's positions (both pages), for this CTA.
struct ChunkScales {
    float f[4][ChunkCfg::BLOCK];          // of the four score accumulators
    float log2f[2], inv[2];               // log2 F and 1 / F of the two pages
    // f_t / F of this CTA's two tiles of values, as two fp16 parts (in the making: first the fifth tile's scale)
    uint32_t value[2][ChunkCfg::BLOCK];
    uint2 key[kPage];                     // g3 and g4 of this CTA's page, as two fp16 parts each (g4's rest kRestUp times)
    int ok[2];                            // the two pages' ids are good
    int pad[2];
};
// The exchange between the threads of a row lies behind the records there.
constexpr int kChunkFp8Xm = ChunkCfg::OFF_REC + ChunkCfg::NREC * (int)sizeof(ChunkScales);
static_assert(kChunkFp8Xm + 256 * 4 <= ChunkCfg::OFF_XM, "position factors exceed their slot");
static_assert(sizeof(ChunkScales) % 16 == 0, "records are read 16 bytes at a time");

// Page `page` of the sequence of a run: its id, -1 (nobody in the tile sees it) or -2 (a bad id).
__device__ __forceinline__ int chunk_page(const ChunkParams& p, const TileRun& s, const int32_t* table, int page) {
    if (page >= p.max_blocks || page * kPage >= s.see) return -1;
    const int id = __ldg(table + page);
    return id >= 0 && id < p.num_blocks ? id : -2;
}

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

}  // namespace dsa
