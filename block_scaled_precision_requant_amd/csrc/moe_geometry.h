// moe_geometry.h -- launch geometry and host-side plans of the expert-layer
// kernels (router, grouped products, 4-bit group GEMV, combine).  Plain C++
// with no HIP header, as bsr_geometry.h.
#pragma once

#include <stdint.h>

#include "bsr_geometry.h"

namespace bsr {

// ---- router ---------------------------------------------------------------
constexpr uint32_t kRouteMaxExperts = 1024;
constexpr uint32_t kRouteMaxTopK = 16;
constexpr uint32_t kRouteThreads = 1024;
constexpr uint32_t kRouteWaves = kRouteThreads / 64;
constexpr uint32_t kRouteMaxBlocks = 256;

// Tokens are cut into `blocks` runs of `per_block`; each run's expert counts
// go to the workspace ([block][expert] u32).  One block needs no workspace.
struct RoutePlan {
    uint32_t blocks, per_block;
    uint64_t bytes;
};

inline RoutePlan moe_route_plan(uint32_t tokens, uint32_t experts) {
    RoutePlan p;
    p.per_block = (uint32_t)div_up(tokens, kRouteMaxBlocks);
    p.per_block = p.per_block < 2 * kRouteWaves ? 2 * kRouteWaves : p.per_block;
    p.blocks = (uint32_t)div_up(tokens, p.per_block);
    p.bytes = p.blocks <= 1 ? 0 : (uint64_t)p.blocks * experts * 4;
    return p;
}

// ---- grouped rows -----------------------------------------------------------
// Row tiles of `bm` rows, none across two experts: at most this many, whatever
// the offsets (each expert with rows adds less than one tile of padding).
inline uint64_t grouped_row_tiles(uint32_t rows, uint32_t experts, uint32_t bm) {
    const uint64_t used = rows < experts ? rows : experts;
    return (rows + used * (bm - 1)) / bm;
}

// ---- 4-bit group GEMV -------------------------------------------------------
// A workgroup owns 16 output columns (with the SiLU product: of the gate and
// of the up half) and up to 16 rows; its waves split K in chunks of 128, taken
// kW4gPass at a time.  Up to kW4gFew rows the passes are twice as long.
constexpr uint32_t kW4gCols = 16;
constexpr uint32_t kW4gRows = 16;
constexpr uint32_t kW4gFew = 4;
constexpr uint32_t kW4gChunk = 128;
constexpr uint32_t kW4gMaxWaves = 16;
#ifndef W4G_TARGET
#define W4G_TARGET 6144
#endif
#ifndef W4G_CT2
#define W4G_CT2 512
#endif

// Chunks per pass, and LDS bytes of one staged activation row (16 bytes of
// padding spread the 16 rows read at one offset over the banks).
BSR_HD constexpr uint32_t w4g_pass(bool few, uint32_t ct) { return few && ct == 1 ? 4 : 2; }
BSR_HD constexpr uint32_t w4g_pitch(uint32_t pass) { return pass * kW4gChunk * 2 + 16; }

struct W4gPlan {
    uint32_t ct;  // column tiles per workgroup (with the SiLU product: a gate and an up tile)
    uint32_t row_tiles, col_tiles, waves, chunks_per_wave, wave_bytes, lds;
};

// The rows of a tile are known only on the device: LDS and passes are sized
// for the most there can be.
inline W4gPlan w4_group_plan(uint32_t rows, uint32_t experts, uint32_t cols, uint32_t k, bool silu) {
    W4gPlan p;
    const uint32_t most = rows < kW4gRows ? rows : kW4gRows;
    const uint32_t chunks = (uint32_t)div_up(k, kW4gChunk);
    p.row_tiles = (uint32_t)grouped_row_tiles(rows, experts, kW4gRows);
    p.ct = silu ? 2 : 1;
    if (!silu && most > kW4gFew && p.row_tiles * div_up(cols, kW4gCols) >= W4G_CT2) p.ct = 2;
    p.col_tiles = (uint32_t)div_up(cols, kW4gCols * (silu ? 1 : p.ct));
    uint64_t waves = div_up(W4G_TARGET, (uint64_t)p.row_tiles * p.col_tiles);
    waves = waves < kW4gMaxWaves ? waves : kW4gMaxWaves;
    waves = waves < chunks ? waves : chunks;
    const uint32_t pass = w4g_pass(most <= kW4gFew, p.ct);
    uint32_t cpw = (uint32_t)div_up(chunks, waves);
    if (cpw > pass) cpw = (uint32_t)div_up(cpw, pass) * pass;  // whole passes
    p.chunks_per_wave = cpw;
    p.waves = (uint32_t)div_up(chunks, cpw);
    const uint32_t few = (most < kW4gFew ? most : kW4gFew) * w4g_pitch(w4g_pass(true, p.ct));
    const uint32_t many = most <= kW4gFew ? 0 : kW4gRows * w4g_pitch(w4g_pass(false, p.ct));
    p.wave_bytes = few > many ? few : many;
    const uint32_t sums = p.waves * 64 * 4 * 4 * p.ct;
    p.lds = p.waves * p.wave_bytes;
    p.lds = p.lds > sums ? p.lds : sums;
    return p;
}

}  // namespace bsr
