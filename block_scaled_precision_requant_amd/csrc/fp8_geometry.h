// fp8_geometry.h -- launch geometry and host-side plans of the FP8 products, the
// weight quantizer and the kernels around sorted tokens.  Plain C++ with no HIP
// header, as bsr_geometry.h.
#pragma once

#include <stdint.h>

#include "bsr_geometry.h"
#include "moe_geometry.h"

namespace bsr {

constexpr uint32_t kFp8Block = 128;       // elements of a scale block, and a stage of K
constexpr uint32_t kFp8MaxK = 1u << 23;   // 256 rows are addressed with 32-bit offsets

inline bool fp8_k_ok(uint32_t k) { return k != 0 && k % kFp8Block == 0 && k < kFp8MaxK; }

// ---- product, tiles through LDS ---------------------------------------------
// 256 x 256 outputs by eight waves of 128 x 64, or 128 x 128 by four of 64 x 64.
constexpr uint32_t kFp8Tall = 256;
constexpr uint32_t kFp8Tile = 128;

// ---- product, operands streamed into registers --------------------------------
// A workgroup owns 16 mt rows by 16 ct columns; its waves split K in chunks of
// 128, kFp8Pass of them in flight.
constexpr uint32_t kFp8Pass = 2;
constexpr uint32_t kFp8MaxWaves = 8;

struct Fp8StreamPlan {
    uint32_t mt, ct, row_tiles, col_tiles, waves, chunks_per_wave, lds;
};

inline Fp8StreamPlan fp8_stream_plan(uint32_t rows, uint32_t experts, uint32_t cols, uint32_t k, bool silu, uint32_t mt,
                                     uint32_t ct) {
    Fp8StreamPlan p;
    p.mt = mt;
    p.ct = ct;
    p.row_tiles = (uint32_t)grouped_row_tiles(rows, experts, 16 * mt);
    p.col_tiles = (uint32_t)div_up(cols, 16 * (silu ? ct / 2 : ct));
    const uint32_t chunks = k / kFp8Block;
    uint64_t waves = 2 * kFp8MaxWaves * (uint64_t)kGemmCus / ((uint64_t)p.row_tiles * p.col_tiles);
    waves = waves > 1 ? waves : 1;
    waves = waves < kFp8MaxWaves ? waves : kFp8MaxWaves;
    waves = waves < chunks ? waves : chunks;
    p.chunks_per_wave = (uint32_t)div_up(chunks, waves);
    p.waves = (uint32_t)div_up(chunks, p.chunks_per_wave);
    p.lds = p.waves * mt * ct * 64 * 16;
    return p;
}

// Which kernel a product runs: streamed (plan) or tiles of `bm` x `bm`.
struct Fp8Choice {
    bool stream;
    Fp8StreamPlan plan;
    uint32_t bm, tiles_m, tiles_n;
    uint64_t threads;
};

inline Fp8Choice fp8_choice(uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, bool silu, bool grouped) {
    Fp8Choice c = {};
    c.stream = rows <= 64 || rows <= 16 * (uint64_t)experts;
    if (c.stream) {
        const uint32_t tiles = grouped ? 1 : (uint32_t)div_up(rows, 16);
        c.plan = fp8_stream_plan(rows, experts, silu ? n / 2 : n, k, silu, tiles > 2 ? 4 : tiles, silu || tiles > 1 ? 2 : 1);
        c.threads = (uint64_t)c.plan.row_tiles * c.plan.col_tiles * c.plan.waves * 64;
        return c;
    }
    c.bm = grouped_row_tiles(rows, experts, kFp8Tall) * div_up(n, kFp8Tall) >= kGemmCus ? kFp8Tall : kFp8Tile;
    c.tiles_m = (uint32_t)grouped_row_tiles(rows, experts, c.bm);
    c.tiles_n = (uint32_t)div_up(n, c.bm);
    c.threads = (uint64_t)c.tiles_m * c.tiles_n * (c.bm == kFp8Tall ? 512 : 256);
    return c;
}

// ---- weight quantizer -----------------------------------------------------------
constexpr uint32_t kQwThreads = 256;

// ---- rows of sorted tokens ------------------------------------------------------
constexpr uint32_t kTokenThreads = 256;

}  // namespace bsr
