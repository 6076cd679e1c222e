// chunk_fp8.cuh -- the operand side of dense attention over an FP8 latent cache:
// codes from global memory to the fp16 operands of the MMAs in shared memory.
//
// What bounds it is no single unit.  Two tokens of 8 sequences of 16K to 128K positions, two tiles of
// 128 rows over 530K positions, take 524 to 551 us.  Of a block's 7830 cycles the issue slots are
// busy in 0.53, the shared-memory pipe in 0.50 with loads and stores (3950 wavefronts a block:
// 1590 loads, 1650 stores, a fifth of them bank conflicts, and barriers) and in 0.26 with the operand
// reads of the MMAs (2020), the tensor pipes in 0.29, and HBM gives 1.1 TB/s.  Most stalls are fixed
// latencies, barriers and branches, then shared memory and instructions that are not there yet.  Over
// an fp16 copy of the cache in global memory, which wrote and read 2304 bytes a position, they
// took 900 us with the copy.  (Many tiles over few positions take the copy: chunk.cu.)
//
// Two teams of CONV_WARPS warps convert, one the keys and one the values, a ring group
// (16 KB of fp16, 8 KB of codes) at a time; the codes of the groups behind are on their way to
// shared memory meanwhile (from L2 for the most part: the factor warps ask for pages up to
// three blocks ahead).  Converting costs 1 instruction per two codes for most keys and 3 for
// values.
//
// Keys: an e4m3 code is exact in fp16, so the products are those of the codes and
// the scores are put together from four accumulators,
//   S = f_0 S_0 + f_1 S_1 + f_2 S_2 + u S_3,
// f_t the scale of tile t (128 elements) of the position, S_t its codes times Q in
// fp32.  The fifth tile, 64 elements, has no accumulator of its own (tensor memory
// is full) and joins S_3, in a unit u of the position's own:
//   u S_3 = f_3 sum c_3 q + f_4 sum c_4 q,   u = f_3 2^j, g3 = f_3 / u = 2^-j, g4 = f_4 / u.
// A scale says nothing of how large its tile's codes are (a tile of zeros has the scale 1), nor of
// how large the queries are that they meet, so neither tile may lose bits to the other: c_3 g3 is
// exact for -7 <= j <= 15 (a code has four bits, 2^-9 to 448; fp16 goes from 2^-24 to 65504), and c_4 g4
// is taken as two fp16 parts, the value rounded and the rest, to 2^-21 of it or 2^-24 u, whichever
// is more.  j is floor(log2 |f_4 / f_3|) - 6, which brings |g4| into [64, 128) (the products end below
// 2^16), and -7 at least, where 2^-24 u is 2^-31 |f_3|.  Past |f_4| = 2^22 |f_3|, j is above 15 and
// c_3 g3 is rounded, to 2^-25 u, which is at most 2^-31 |f_4|.
//
// Values: code * f_t / F, one rounding to fp16, with F the power of two that brings
// the largest value scale of the page's positions into [64, 128), so that values end
// below 2^16 (codes end at 448); positions behind the sequence's end do not count,
// whatever they hold.  The weights that multiply them are P F (the softmax adds log2 F to the
// scores and divides F out of the sums).
#pragma once
#include <cuda_fp16.h>

#include "chunk_cfg.cuh"

namespace dsa {

// A value as two fp16 parts, the rounded value (low) and the rest times `up`.
__device__ __forceinline__ uint32_t two_halves(float v, float up = 1.0f) {
    const __half h = __float2half_rn(v), l = __float2half_rn((v - __half2float(h)) * up);
    return (uint32_t)__half_as_ushort(h) | (uint32_t)__half_as_ushort(l) << 16;
}
// The rest of g4 is stored 2^10 times as large and meets codes 2^10 times as small (exact), so that it
// does not lose bits to fp16's smallest step before it is multiplied by a code of up to 448.
constexpr float kRestUp = 1024.0f;

// The unit of tiles 3 and 4 of a position, and their scales in it.  Magnitudes compare as integers, and
// their difference shifted by the mantissa's width is floor(log2 |f4 / f3|) of normal numbers.
struct Fp8Unit {
    float u, g3, g4;
};
__device__ __forceinline__ Fp8Unit fp8_unit(float f3, float f4) {
    const int b3 = (int)(__float_as_uint(f3) & 0x7FFFFFFFu), b4 = (int)(__float_as_uint(f4) & 0x7FFFFFFFu);
    Fp8Unit t;
    constexpr int kTiny = 27 << 23;                      // 2^-100
    if (b3 >= kTiny && b3 < 0x7F800000) {
        const int d = ((b4 - b3) >> 23) - 6, j = d < -7 ? -7 : d;
        t.u = __uint_as_float(__float_as_uint(f3) + ((uint32_t)j << 23));
        t.g3 = j > 60 ? 0.0f : __uint_as_float((uint32_t)(127 - j) << 23);
        t.g4 = f4 / t.u;
    } else if (b3 < kTiny) {                             // nothing beside any f4 to be met
        t.u = __uint_as_float((uint32_t)((b4 < kTiny ? kTiny : b4) - (6 << 23)) & 0x7F800000u);
        t.g3 = f3 / t.u;
        t.g4 = f4 / t.u;
    } else {                                             // infinite or NaN: the score is, whatever the codes
        t.u = f3;
        t.g3 = 1.0f;
        t.g4 = 0.0f;
    }
    return t;
}

// The factors of the positions of page `half` of every block: a warp each, two positions a lane.
__device__ __forceinline__ bool fp8_factors(const ChunkParams& p, ChunkMisc* m, ChunkScales* ring, int half, uint32_t crank,
                                            volatile int* abort, uint64_t wlim) {
    using Cfg = ChunkCfg;
    const int lane = threadIdx.x & 31;
    uint32_t rr = 0, ph = 1;
    bool bad = false, ok = true;
#pragma unroll 1
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
        const int32_t* table = p.block_table + (int64_t)sg.b * p.max_blocks;
        int id = -1;
        float raw[2][Cfg::TILES];          // of the next block
#pragma unroll 1
        for (int k = sg.k0 - 1; k < sg.k1; ++k) {
            const int page = id;
            float log2f = 0.0f, inv = 1.0f;
            ChunkScales& rec = ring[rr];
            if (k >= sg.k0) {
                if (!warp_wait(&m->rec_empty[rr], ph, abort, wlim)) {
                    ok = false;
                    break;
                }
                bad = bad || page == -2;
                float top = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int pos = 64 * half + 32 * i + lane;
                    const bool seen = k * Cfg::BLOCK + pos < sg.see;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        rec.f[t][pos] = raw[i][t];
                        if (seen) top = fmaxf(top, fabsf(raw[i][t]));
                    }
                    rec.value[0][pos] = __float_as_uint(raw[i][4]);
                }
                // magnitudes compare as integers
                const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
                int E = (int)(bits >> 23) - 127;
                E = bits == 0 ? 6 : E < -100 ? -100 : E > 120 ? 120 : E;
                log2f = (float)(E - 6);
                inv = __uint_as_float((uint32_t)(6 - E + 127) << 23);
            }
            if (k + 1 < sg.k1) {
                id = chunk_page(p, sg, table, 2 * (k + 1) + half);
                const float* src = p.kv_scale + (int64_t)(id < 0 ? 0 : id) * kPage * Cfg::TILES;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int t = 0; t < Cfg::TILES; ++t)
                        raw[i][t] = id < 0 ? 0.0f : __ldg(src + (32 * i + lane) * Cfg::TILES + t);
                // the whole page in L2, by the CTA that takes it as keys
                if (lane == 0 && id >= 0 && half == (int)crank)
                    prefetch_l2(p.codes + (int64_t)id * kPage * kDqk, kPage * kDqk);
            }
            if (k < sg.k0) continue;
#pragma unroll 1
            for (int pos = 64 * half + lane; pos < 64 * half + 64; pos += 32) {
                const float f3 = rec.f[3][pos], f4 = __uint_as_float(rec.value[0][pos]);
                const Fp8Unit t = fp8_unit(f3, f4);
                rec.f[3][pos] = t.u;
                if (half == (int)crank) rec.key[pos & (kPage - 1)] = make_uint2(two_halves(t.g3, 1.0f), two_halves(t.g4, kRestUp));
                rec.value[0][pos] = two_halves(rec.f[2 * crank][pos] * inv);
                rec.value[1][pos] = two_halves((crank == 0 ? rec.f[1][pos] : f3) * inv);
            }
            if (lane == 0) {
                rec.log2f[half] = log2f;
                rec.inv[half] = inv;
                rec.ok[half] = page != -2;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&m->rec_full[rr]);
            if (++rr == Cfg::NREC) {
                rr = 0;
                ph ^= 1;
            }
        }
    }
    if (bad && lane == 0) atomicCAS(p.status, 0u, (uint32_t)kStBounds);
    return ok;
}

// 16 codes as fp16 (exact).
__device__ __forceinline__ void widen16(uint4 raw, __half2 (&h)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t x;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)(w[i >> 1] >> (16 * (i & 1)))));
        h[i] = *reinterpret_cast<const __half2*>(&x);
    }
}
// Two neighbouring 16-byte pieces of a 128-byte operand row: `at` is the place of the first,
// an even one before the swizzle.
__device__ __forceinline__ void put16(uint32_t at, const __half2 (&h)[8]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&h[0]);
    st_shared_v4(at, make_uint4(w[0], w[1], w[2], w[3]));
    st_shared_v4(at ^ 16u, make_uint4(w[4], w[5], w[6], w[7]));
}
__device__ __forceinline__ __half2 low_half(uint32_t two) {
    const __half2 v = *reinterpret_cast<const __half2*>(&two);
    return __half2half2(__low2half(v));
}
__device__ __forceinline__ __half2 high_half(uint32_t two) {
    const __half2 v = *reinterpret_cast<const __half2*>(&two);
    return __half2half2(__high2half(v));
}

// Loads of codes, of keys or of values (a warp each; one elected lane acts): a ring slot for the
// codes of every slot of the operand ring.  They land on the barrier that the slot's MMAs
// complete on, so that the converters wait once for both.
__device__ __forceinline__ bool fp8_codes(const ChunkParams& p, ChunkMisc* m, uint8_t* smem, const CUtensorMap& tm_k,
                                          const CUtensorMap& tm_r, const CUtensorMap& tm_v, bool keys, uint32_t crank,
                                          volatile int* abort, uint64_t wlim) {
    using Cfg = ChunkCfg;
    const bool el = elect_one();
    uint8_t* codes = smem + (keys ? Cfg::OFF_KC : Cfg::OFF_VC);
    uint64_t* full = keys ? m->k_empty : m->v_empty;
    uint64_t* empty = keys ? m->kc_empty : m->vc_empty;
    const uint32_t slots = keys ? Cfg::FKRING : Cfg::FVRING;
    uint32_t cr = 0, ph = 1;
#pragma unroll 1
    for (int ns = 0;; ++ns) {
        const int sr = ns % Cfg::NSEG;
        if (!elected_wait(el, &m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim)) return false;
        const TileRun sg = m->seg[sr];
        __syncwarp();
        if (el) mbar_arrive(&m->seg_empty[sr]);
        if (sg.b < 0) return true;
        const int32_t* table = p.block_table + (int64_t)sg.b * p.max_blocks;
        const int k0 = __shfl_sync(0xffffffffu, sg.k0, 0), k1 = __shfl_sync(0xffffffffu, sg.k1, 0);
        int id0 = chunk_page(p, sg, table, 2 * k0), id1 = chunk_page(p, sg, table, 2 * k0 + 1);
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
            const int next0 = chunk_page(p, sg, table, 2 * k + 2), next1 = chunk_page(p, sg, table, 2 * k + 3);
            const int groups = keys ? 5 : chunk_block(sg, k).ngroups;
#pragma unroll 1
            for (int g = 0; g < groups; ++g) {
                if (!elected_wait(el, &empty[cr], ph, abort, wlim)) return false;
                const int id = (keys ? crank == 0 : g < 2) ? id0 : id1;
                const bool last = keys && g == 0;        // the fifth tile
                if (el) {
                    uint8_t* dst = codes + cr * Cfg::CGROUP;
                    // (a page that is not there: whatever the ring holds is replaced later)
                    if (id < 0) mbar_arrive(&full[cr]);
                    else mbar_arrive_expect_tx(&full[cr], last ? Cfg::CGROUP / 2 : Cfg::CGROUP);
                    if (id >= 0) {
                        const int x = !keys ? 256 * (int)crank : 128 * (g == 0 ? 4 : g == 1 ? 3 : g - 2);
                        const int y = id * kPage + (keys ? 0 : 32 * (g & 1));
                        tma_load_2d(dst, !keys ? &tm_v : last ? &tm_r : &tm_k, &full[cr], x, y);
                    }
                }
                if (++cr == slots) {
                    cr = 0;
                    ph ^= 1;
                }
            }
            id0 = next0;
            id1 = next1;
        }
    }
}

// Keys of this CTA's page of every block: groups in the order fifth tile (rests, then
// values: the small ones first), tile 3, tiles 0 to 2; each two chunks of [64 rows x 64].
// A thread takes 16 codes at a time; eight neighbouring lanes take four pieces of two rows,
// of different halves of the 128, which keeps both their reads and their writes on
// different banks.  The loops over groups are rolled: unrolled code of this many roles does not
// fit the instruction cache, and ran at half of this speed.
__device__ __forceinline__ bool fp8_keys(const ChunkParams& p, ChunkMisc* m, uint8_t* smem, int ti, uint32_t crank,
                                         volatile int* abort, uint64_t wlim) {
    using Cfg = ChunkCfg;
    constexpr int CW = Cfg::CONV_WARPS, THREADS = 32 * CW, N = 16 / CW, NR = 8 / CW;
    const ChunkScales* ring = reinterpret_cast<const ChunkScales*>(smem + Cfg::OFF_REC);
    uint8_t* codes = smem + Cfg::OFF_KC;
    const int lane = ti & 31, bit = (lane >> 2) & 1;
    const int q = (lane & 3) | ((((lane >> 3) & 1) ^ bit) << 2), row = 2 * (ti >> 4) + bit;
    const int rq = lane & 3, rrow = ti >> 2;             // of the fifth tile's 64 codes
    const uint32_t src = smem_u32(codes) + row * 128 + 16 * q, rsrc = smem_u32(codes) + rrow * 64 + 16 * rq;
    const uint32_t keys = smem_u32(smem + Cfg::OFF_FK);
    const uint32_t dst = keys + (q >> 2) * 8192 + row * 128 + (((2 * (q & 3)) ^ (row & 7)) << 4);
    const uint32_t rdst = keys + rrow * 128 + (((2 * rq) ^ (rrow & 7)) << 4);
    uint32_t rr = 0, rph = 0, r = 0, ph = 0;
#pragma unroll 1
    for (int ns = 0;; ++ns) {
        const int sr = ns % Cfg::NSEG;
        if (!warp_wait(&m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim)) return false;
        const TileRun sg = m->seg[sr];
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->seg_empty[sr]);
        if (sg.b < 0) return true;
#pragma unroll 1
        for (int k = sg.k0; k < sg.k1; ++k) {
            const ChunkScales& rec = ring[rr];
            bool ok = warp_wait(&m->rec_full[rr], rph, abort, wlim);
#pragma unroll 1
            for (int g = 0; g < 5; ++g) {
                ok = ok && warp_wait(&m->k_empty[r], ph, abort, wlim);
                if (ok) {
                    const uint32_t off = r * Cfg::CGROUP, to = r * Cfg::FGROUP;
                    if (g == 0) {
#pragma unroll 1
                        for (int j = 0; j < NR; ++j) {
                            const uint32_t f = rec.key[rrow + j * 8 * CW].y;
                            const __half2 gh = low_half(f), gl = high_half(f), down = __float2half2_rn(1.0f / kRestUp);
                            __half2 h[8], l[8];
                            widen16(ld_shared_v4(rsrc + off + j * (8 * CW * 64)), h);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const __half2 c = h[e];
                                h[e] = __hmul2(c, gh);
                                l[e] = __hfma2(__hmul2(c, down), gl, __hfma2(c, gh, __hneg2(h[e])));
                            }
                            put16(rdst + to + j * (8 * CW * 128), l);
                            put16(rdst + to + j * (8 * CW * 128) + 8192, h);
                        }
                    } else {
                        __half2 f[N];
#pragma unroll
                        for (int j = 0; j < N; ++j) f[j] = low_half(g == 1 ? rec.key[row + j * 4 * CW].x : 0x3C00u);
                        uint4 v[N];
#pragma unroll
                        for (int j = 0; j < N; ++j) v[j] = ld_shared_v4(src + off + j * (4 * CW * 128));
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            __half2 h[8];
                            widen16(v[j], h);
#pragma unroll
                            for (int e = 0; e < 8; ++e) h[e] = __hmul2(h[e], f[j]);
                            put16(dst + to + j * (4 * CW * 128), h);
                        }
                    }
                }
                fence_proxy_async_smem();
                ok = named_bar_and(2, THREADS, ok);
                if (!ok) return false;
                if (ti == 0) {
                    arrive_leader(&m->k_full[r], crank);
                    mbar_arrive(&m->kc_empty[r]);
                    if (g == 1) mbar_arrive(&m->rec_empty[rr]);
                }
                if (++r == Cfg::FKRING) {
                    r = 0;
                    ph ^= 1;
                }
            }
            if (++rr == Cfg::NREC) {
                rr = 0;
                rph ^= 1;
            }
        }
    }
}

// Values: this CTA's 256 of the 512 columns of both pages, in groups of 32 positions (four
// chunks of [32 rows x 64]).  Positions that nobody in the tile sees become zeros, and so do
// non-finite values of positions that only some of its tokens see (a weight of zero still
// multiplies the value; the tokens that see it have a non-finite score already).
__device__ __forceinline__ bool fp8_values(const ChunkParams& p, ChunkMisc* m, uint8_t* smem, int ti, uint32_t crank,
                                           volatile int* abort, uint64_t wlim) {
    using Cfg = ChunkCfg;
    constexpr int CW = Cfg::CONV_WARPS, THREADS = 32 * CW, N = 16 / CW;
    const ChunkScales* ring = reinterpret_cast<const ChunkScales*>(smem + Cfg::OFF_REC);
    uint8_t* codes = smem + Cfg::OFF_VC;
    const int lane = ti & 31, bit = (lane >> 2) & 1;
    const int q = (lane & 3) | ((((lane >> 3) & 1) ^ bit) << 2) | ((lane >> 4) << 3), row = 2 * (ti >> 5) + bit;
    const uint32_t src = smem_u32(codes) + row * 256 + 16 * q;
    const uint32_t dst = smem_u32(smem + Cfg::OFF_FV) + (q >> 2) * 4096 + row * 128 + (((2 * (q & 3)) ^ (row & 7)) << 4);
    static_assert(2 * CW % 8 == 0, "a thread's rows lie a multiple of eight apart: one place in the swizzle");
    uint32_t rr = 0, rph = 0, r = 0, ph = 0;
#pragma unroll 1
    for (int ns = 0;; ++ns) {
        const int sr = ns % Cfg::NSEG;
        if (!warp_wait(&m->seg_full[sr], (ns / Cfg::NSEG) & 1, abort, wlim)) return false;
        const TileRun sg = m->seg[sr];
        __syncwarp();
        if (lane == 0) mbar_arrive(&m->seg_empty[sr]);
        if (sg.b < 0) return true;
        const int32_t* table = p.block_table + (int64_t)sg.b * p.max_blocks;
        auto page = [&](int i) { return i < 2 * sg.k1 ? chunk_page(p, sg, table, i) : -1; };
        int id0 = page(2 * sg.k0), id1 = page(2 * sg.k0 + 1);
#pragma unroll 1
        for (int k = sg.k0; k < sg.k1; ++k) {
            const int next0 = page(2 * k + 2), next1 = page(2 * k + 3);
            const ChunkBlock cb = chunk_block(sg, k);
            const ChunkScales& rec = ring[rr];
            bool ok = warp_wait(&m->rec_full[rr], rph, abort, wlim);
#pragma unroll 1
            for (int g = 0; g < cb.ngroups; ++g) {
                const int id = g < 2 ? id0 : id1;
                ok = ok && warp_wait(&m->v_empty[r], ph, abort, wlim);
                if (ok) {
                    const bool edge = g >= cb.fix_from || id < 0;
                    const uint32_t from = src + r * Cfg::CGROUP, to = dst + r * Cfg::FGROUP;
                    uint32_t f[N];
                    uint4 v[N];
#pragma unroll
                    for (int j = 0; j < N; ++j) f[j] = rec.value[q >> 3][32 * g + row + j * 2 * CW];
#pragma unroll
                    for (int j = 0; j < N; ++j) v[j] = ld_shared_v4(from + j * (2 * CW * 256));
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        const __half2 fh = low_half(f[j]), fl = high_half(f[j]);
                        __half2 h[8];
                        widen16(v[j], h);
#pragma unroll
                        for (int e = 0; e < 8; ++e) h[e] = __hfma2(h[e], fh, __hmul2(h[e], fl));
                        put16(to + j * (2 * CW * 128), h);
                    }
                    if (edge) {
                        // this thread's pieces once more
#pragma unroll 1
                        for (int j = 0; j < 2 * N; ++j) {
                            const int rw = row + (j >> 1) * 2 * CW, pos = k * Cfg::BLOCK + 32 * g + rw;
                            uint32_t* at = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_FV + r * Cfg::FGROUP + (q >> 2) * 4096 +
                                                                       rw * 128 + (((2 * (q & 3) + (j & 1)) ^ (rw & 7)) << 4));
                            const bool none = id < 0 || pos >= sg.see, some = pos >= sg.see_all;
#pragma unroll 1
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t w = at[e];
                                const bool odd = (w & 0x7C00u) == 0x7C00u || (w & 0x7C000000u) == 0x7C000000u;
                                if (none || (some && odd)) at[e] = 0u;
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                ok = named_bar_and(3, THREADS, ok);
                if (!ok) return false;
                if (ti == 0) {
                    arrive_leader(&m->v_full[r], crank);
                    mbar_arrive(&m->vc_empty[r]);
                    if (g + 1 == cb.ngroups) mbar_arrive(&m->rec_empty[rr]);
                }
                if (++r == Cfg::FVRING) {
                    r = 0;
                    ph ^= 1;
                }
            }
            if (!ok) return false;
            if (++rr == Cfg::NREC) {
                rr = 0;
                rph ^= 1;
            }
            id0 = next0;
            id1 = next1;
        }
    }
}

}  // namespace dsa
