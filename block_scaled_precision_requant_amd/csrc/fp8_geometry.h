// fp8_geometry.h -- launch geometry and host-side plans of the FP8 products, the
// weight quantizer and the kernels around sorted tokens.  Plain C++ with no HIP
// header, as bsr_geometry.h.
#pragma once

#include <stdint.h>

#include "bsr_geometry.h"
#include "moe_geometry.h"

namespace bsr {

constexpr uint32_t kFp8Block = 128;       // elements of a scale block, and a stage of K
constexpr uint32_t kFp8MaxK = 1u << 23;   // the rows of a tile are addressed with 32-bit offsets

inline bool fp8_k_ok(uint32_t k) { return k != 0 && k % kFp8Block == 0 && k < kFp8MaxK; }

// ---- product, tiles through LDS ---------------------------------------------
// Shapes of a workgroup's tile, in the order of kFp8Shapes.  `cost`: tenths of a
// microsecond that one round of workgroups on every CU takes at k = 4096 (MI355X, the
// weight in the cache behind the L2, one call behind the other from the host, of which none
// takes less than 6.5); `last`: the same where a last round leaves half of the places
// empty.  They serve to order the shapes.  In captured graphs the rounds take 51 (half empty
// 39), 47, 61, 122; 49, 52, 72, 161; 62, 71, 105, 162; 140, 218, 367, 590, the pair 367 (301).
// Over 330 sizes of 5 to 8192 rows, the weight in the cache and past it, the shape taken is
// 1.3 % behind the best of the 17 on average, 24 % at most (64 rows, n 4096, k 14336: 64 x 16
// 18.7 us, 32 x 32 15.1).  64 x 128 is counted once a CU although two fit: counted twice
// (242, half empty 162) the average is 2.6 %, and 300 x 8192 x 8192 (past
// the cache) would take it at 53 us instead of 128 x 128 at 36.
struct Fp8Shape {
    uint16_t bm, bn, threads, per_cu, cost, last;
};
constexpr uint32_t kFp8NumShapes = 16;
constexpr Fp8Shape kFp8Shapes[kFp8NumShapes] = {
    {16, 16, 256, 2, 66, 65},     {16, 32, 256, 1, 66, 66},    {16, 64, 256, 1, 87, 87},    {16, 128, 256, 1, 142, 142},
    {32, 16, 256, 1, 66, 66},     {32, 32, 256, 1, 72, 72},    {32, 64, 256, 1, 102, 102},  {32, 128, 192, 1, 158, 158},
    {64, 16, 256, 1, 71, 71},     {64, 32, 256, 1, 84, 84},    {64, 64, 256, 1, 116, 116},  {64, 128, 256, 1, 170, 170},
    {128, 64, 512, 1, 160, 160},  {128, 128, 512, 1, 243, 243}, {256, 128, 512, 1, 404, 404}, {256, 256, 512, 1, 530, 530},
};
// Two workgroups of 128 x 128 by four waves a CU, where there are tiles for more than a
// round of every larger shape: an entry of its own, since the tile is the same.
constexpr Fp8Shape kFp8Pair = {128, 128, 256, 2, 405, 245};
constexpr uint32_t kFp8PairIndex = kFp8NumShapes;
BSR_HD constexpr Fp8Shape fp8_shape(uint32_t i) { return i == kFp8PairIndex ? kFp8Pair : kFp8Shapes[i]; }

// ---- product, the weight streamed into registers ------------------------------
// A workgroup owns 16 rows by 16 columns (and as many of the up half); its waves split K
// in chunks of 128, two of them in flight.
constexpr uint32_t kFp8MaxWaves = 8;
constexpr uint32_t kFp8Few = 4;  // rows (of an expert, on average) up to which it runs

struct Fp8StreamPlan {
    uint32_t row_tiles, col_tiles, waves, chunks_per_wave, lds;
};

inline Fp8StreamPlan fp8_stream_plan(uint32_t rows, uint32_t experts, uint32_t cols, uint32_t k, bool silu) {
    Fp8StreamPlan p;
    p.row_tiles = (uint32_t)grouped_row_tiles(rows, experts, 16);
    p.col_tiles = (uint32_t)div_up(cols, 16);
    const uint32_t chunks = k / kFp8Block;
    uint64_t waves = 2 * kFp8MaxWaves * (uint64_t)kGemmCus / ((uint64_t)p.row_tiles * p.col_tiles);
    waves = waves > 1 ? waves : 1;
    waves = waves < kFp8MaxWaves ? waves : kFp8MaxWaves;
    waves = waves < chunks ? waves : chunks;
    p.chunks_per_wave = (uint32_t)div_up(chunks, waves);
    p.waves = (uint32_t)div_up(chunks, p.chunks_per_wave);
    p.lds = p.waves * (silu ? 2 : 1) * 64 * 16;
    return p;
}

// Which kernel a product runs: streamed (plan), or tiles of shape `shape`.
struct Fp8Choice {
    bool stream;
    Fp8StreamPlan plan;
    uint32_t shape, tiles_m, tiles_n;
    uint64_t threads;
};

// Rounds of workgroups that shape i takes for `tiles` tiles, by their cost.
inline uint64_t fp8_cost(uint32_t i, uint64_t tiles) {
    const Fp8Shape f = fp8_shape(i);
    const uint64_t slots = (uint64_t)f.per_cu * kGemmCus, left = tiles % slots;
    return tiles / slots * f.cost + (left == 0 ? 0 : (2 * left <= slots ? f.last : f.cost));
}

// Row tiles of shape i that `rows` rows of `used` experts make, as far as the host can
// say: each expert leaves half a tile empty.
inline uint64_t fp8_expected_tiles(uint32_t i, uint32_t rows, uint64_t used) {
    const uint32_t bm = fp8_shape(i).bm;
    if (used == 1) return div_up(rows, bm);
    const uint64_t tiles = (2 * (uint64_t)rows + used * bm) / (2 * bm);
    return tiles > used ? tiles : used;
}

// Up to kFp8Few rows (of an expert) the weight alone is read, streamed.  Both sides (us;
// weights past the cache; 1 / 4 / 5 rows, streamed and the best tiles): n 28672, k 4096 24.0 /
// 23.9 / 24.5, 16 x 128 24.6 throughout; n 4096, k 14336 13.7 / 13.1 / 13.3, 16 x 16 13.6 / 13.1 /
// 13.0; n 28672, k 256 5.0 / 5.3 / 5.3, 5.4; n 28672, k 8192 50 / 48 / -, 16 x 16 44 / 43 / -; 64
// experts of 1 / 4 / 5 / 8 rows, n 4096, k 2048 93 / 92 / 93 / 98, 64 x 128 90 / 91 / 91 / 92; 32,
// n 2048, k 4096 55 / 54 / 55 / 63, 63 throughout.
// Else the shape whose rounds cost least: one round on all CUs if any shape has one, so that
// for few rows the columns, for many the tile's area, are what grows.  Measured against its
// neighbours (us; rows, n, k; the chosen shape first; the weight in the cache): 16, 4096,
// 14336: 16 x 16 12.0, 16 x 32 12.2, 32 x 32 13.8; 256, 4096, 4096: 64 x 64 11.1, 128 x 64
// 12.6, 64 x 32 13.6; 512, 4096, 14336: 128 x 64 40.5, 64 x 128 48, 128 x 128 56; 128, 28672,
// 8192: 128 x 128 39.5, 64 x 128 42.8; 1024, 14336, 4096: 256 x 256 54, pairs 63; 2048, 4096,
// 14336, past the cache: 256 x 128 120, pairs 136.
// Several experts with tiles for most of the CUs go by their rows on average, since
// reading the weights is most of the time and wide tiles read them best: 64 x 128 below
// 32, 256 x 128 below 96 or while 256 x 256 has less than two rounds, else 256 x 256.  Both
// sides, even and (uneven) counts: 64 experts of 8, n 4096, k 2048: 64 x 128 92 (91), 256 x 128
// 104 (104), 32 x 128 118 (118).  Of 32: 64 x 128 96 (103), 256 x 128 110 (111); 16 of 32, n
// 8192, k 4096: 121 (129), 134 (120).  Of 64: 122 (146), 136 (118), so the border stands where
// uneven counts turn.  64 of 96, n 4096, k 2048: 256 x 128 130 (136), 256 x 256 134 (136); of
// 160: 171 (175), 163 (169); of 512: 353 (392), 286 (336); of 16 of 96, n 8192, k 4096, 138 (143),
// 144 (176).
// (128 x 64, whose two groups copy little each, is left to one weight: 3234 rows of 64
// experts, n 256, k 7808: 55 us against 46 of 64 x 128.)
inline Fp8Choice fp8_choice(uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, bool silu) {
    Fp8Choice c = {};
    const uint64_t used = rows < experts ? rows : experts;
    c.stream = rows <= kFp8Few * used;
    if (c.stream) {
        c.plan = fp8_stream_plan(rows, experts, silu ? n / 2 : n, k, silu);
        c.threads = (uint64_t)c.plan.row_tiles * c.plan.col_tiles * c.plan.waves * 64;
        return c;
    }
    constexpr uint32_t k64x128 = 11, k128x64 = 12, k256x128 = 14, k256x256 = 15;
    auto tiles = [&](uint32_t i) { return fp8_expected_tiles(i, rows, used) * div_up(n, fp8_shape(i).bn); };
    bool by_rows = false;
    if (used > 1) {
        c.shape = rows < 32 * used ? k64x128
                                   : (rows < 96 * used || tiles(k256x256) < 2 * kGemmCus ? k256x128 : k256x256);
        by_rows = 4 * tiles(c.shape) >= 3 * kGemmCus;
    }
    if (!by_rows) {
        uint64_t best = ~0ull;
        for (uint32_t i = 0; i <= kFp8PairIndex; ++i) {
            if ((silu && fp8_shape(i).bn == 16) || (used > 1 && i == k128x64)) continue;
            const uint64_t cost = fp8_cost(i, tiles(i));
            if (cost <= best) {  // (of equal ones the larger tile)
                best = cost;
                c.shape = i;
            }
        }
    }
    const Fp8Shape f = fp8_shape(c.shape);
    c.tiles_m = (uint32_t)grouped_row_tiles(rows, experts, f.bm);
    c.tiles_n = (uint32_t)div_up(n, f.bn);
    c.threads = (uint64_t)c.tiles_m * c.tiles_n * f.threads;
    return c;
}

// ---- weight quantizer -----------------------------------------------------------
constexpr uint32_t kQwThreads = 256;

// ---- rows of sorted tokens ------------------------------------------------------
constexpr uint32_t kTokenThreads = 256;

}  // namespace bsr
