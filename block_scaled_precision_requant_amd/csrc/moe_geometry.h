// moe_geometry.h -- launch geometry and host-side plans of the expert-layer
// kernels (router, grouped products, 4-bit group GEMV, combine).  Plain C++
// with no HIP header, as bsr_geometry.h.  Times at the rules: a pass in a captured
// graph whose inputs rotate past 512 MB, so that weights come from HBM.
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
// One workgroup alone takes up to this many tokens; more go in runs of 32 at least.
// Alone and in two launches: 64 tokens of 64 experts, top 8, 5.9 and 7.9 us, of 256
// 11.5 and 10.3, of 1024 41.5 and 27.1; 128 tokens of 128, top 4, 9.5 and 8.1.
constexpr uint32_t kRouteAlone = 64;

// Tokens are cut into `blocks` runs of `per_block`; each run's expert counts
// go to the workspace ([block][pitch] u32, a pitch of whole 16 bytes; in all at
// most 1024 bytes per expert).  One block needs no workspace.
struct RoutePlan {
    uint32_t blocks, per_block;
    uint64_t bytes;
};
BSR_HD constexpr uint32_t route_pitch(uint32_t experts) { return (experts + 3) & ~3u; }

inline RoutePlan moe_route_plan(uint32_t tokens, uint32_t experts) {
    RoutePlan p;
    const uint32_t most = kRouteMaxBlocks * experts / route_pitch(experts);
    p.per_block = (uint32_t)div_up(tokens, most);
    p.per_block = p.per_block < 2 * kRouteWaves ? 2 * kRouteWaves : p.per_block;
    if (tokens <= kRouteAlone) p.per_block = kRouteAlone;
    p.blocks = (uint32_t)div_up(tokens, p.per_block);
    p.bytes = p.blocks <= 1 ? 0 : (uint64_t)p.blocks * route_pitch(experts) * 4;
    return p;
}

// ---- grouped rows -----------------------------------------------------------
// Row tiles of `bm` rows, none across two experts: at most this many, whatever
// the offsets (each expert with rows adds less than one tile of padding).
inline uint64_t grouped_row_tiles(uint32_t rows, uint32_t experts, uint32_t bm) {
    const uint64_t used = rows < experts ? rows : experts;
    return (rows + used * (bm - 1)) / bm;
}

// A launch has fewer than 2^32 threads.
constexpr uint64_t kMaxThreads = (1ull << 32) - 1;

// ---- combine ----------------------------------------------------------------
constexpr uint32_t kCombineThreads = 256;

// ---- grouped GEMV (few rows per expert) -------------------------------------
// A workgroup owns 16 output columns and a tile of up to 16 rows, or 4; its
// waves split K in chunks of 128 bytes, two to a pass.
constexpr uint32_t kGgCols = 16;
constexpr uint32_t kGgRows = 16;
constexpr uint32_t kGgFew = 4;
constexpr uint32_t kGgChunk = 128;
constexpr uint32_t kGgPass = 2;
// 16 waves leave a wave 128 registers, which tiles of 4 rows fit.
BSR_HD constexpr uint32_t gg_max_waves(uint32_t rows) { return rows <= kGgFew ? 16 : 8; }
// LDS bytes of a wave: its pass's activation rows (16 bytes of padding spread
// 16 rows over the banks) and their scales, [block][row].
BSR_HD constexpr uint32_t gg_pitch() { return kGgPass * kGgChunk + 16; }
BSR_HD constexpr uint32_t gg_wave_bytes(uint32_t rows) { return rows * (gg_pitch() + kGgPass * 4 * 4); }

// The GEMV runs for one row per used expert on average, and for more while the
// GEMM's 128 x 128 tiles would leave CUs idle.  Measured with the same rows for every
// expert (GEMV against GEMM, us; experts, n, k): 8, 4096, 14336 at 1 / 4 / 8 / 16 rows each
// 101 / 112 / 124 / 148 against 119 / 125 / 126 / 127; 16, 512, 4096 at 1 / 16 rows 11.5 /
// 13.8 against 30 / 31; 64, 4096, 2048 at 1 / 2 / 4 rows 105 / 110 / 122 against 117 / 118 / 120.
// K is not looked at: small grids of a long K are left to the GEMM although the GEMV's
// split of K suits them (8, 256, 7200 at 74 rows 25 against 100).
inline bool grouped_gemv_rule(uint32_t rows, uint32_t experts, uint32_t n) {
    const uint64_t used = rows < experts ? rows : experts;
    const uint64_t tiles = grouped_row_tiles(rows, experts, kGemmBM) * div_up(n, kGemmBN);
    return rows <= used || rows * tiles <= 6 * kGemmCus * used;
}

struct GroupedGemvPlan {
    uint32_t rows, row_tiles, col_tiles, waves, chunks_per_wave, lds;
};

inline GroupedGemvPlan grouped_gemv_plan(uint32_t rows, uint32_t experts, uint32_t n, uint32_t k) {
    GroupedGemvPlan p;
    const uint32_t used = rows < experts ? rows : experts;
    p.rows = rows <= kGgFew || rows <= 2 * (uint64_t)used ? kGgFew : kGgRows;
    const uint32_t chunks = (uint32_t)div_up(k, kGgChunk);
    p.row_tiles = (uint32_t)grouped_row_tiles(rows, experts, p.rows);
    p.col_tiles = (uint32_t)div_up(n, kGgCols);
    const uint32_t most = gg_max_waves(p.rows);
    uint64_t waves = most * (uint64_t)kGemmCus / ((uint64_t)p.row_tiles * p.col_tiles);  // what runs at once
    waves = waves > 1 ? waves : 1;
    waves = waves < most ? waves : most;
    waves = waves < chunks ? waves : chunks;
    p.chunks_per_wave = (uint32_t)div_up(div_up(chunks, waves), kGgPass) * kGgPass;  // whole passes
    p.waves = (uint32_t)div_up(chunks, p.chunks_per_wave);
    p.lds = p.waves * gg_wave_bytes(p.rows);
    const uint32_t sums = p.waves * 64 * 4 * 4;
    p.lds = p.lds > sums ? p.lds : sums;
    return p;
}

// Threads of a grouped launch (its 16-row tiles below 2^31).
inline uint64_t grouped_threads(uint32_t rows, uint32_t experts, uint32_t n, uint32_t k) {
    if (!grouped_gemv_rule(rows, experts, n)) return grouped_row_tiles(rows, experts, kGemmBM) * div_up(n, kGemmBN) * 256;
    const GroupedGemvPlan p = grouped_gemv_plan(rows, experts, n, k);
    return (uint64_t)p.row_tiles * p.col_tiles * p.waves * 64;
}

// ---- 4-bit group GEMV -------------------------------------------------------
// A workgroup owns a tile of up to 16 rows, or 4, and 16 output columns, 32
// (`ct` tiles of 16), or with the SiLU product 16 of the gate and 16 of the up
// half; its waves split K in chunks of 128, several to a pass.
constexpr uint32_t kW4gCols = 16;
constexpr uint32_t kW4gRows = 16;
constexpr uint32_t kW4gFew = 4;
constexpr uint32_t kW4gChunk = 128;

// gpc: groups per chunk (0: one scale per weight row).
// Chunks per pass: the weights in flight per wave, as many as the registers
// hold beside the scales of a group of 32 and, from 5 rows on, the activations.
BSR_HD constexpr uint32_t w4g_pass(uint32_t ct, uint32_t gpc) { return ct == 2 || gpc == 4 ? 2 : 4; }
// Chunks per staging of the activations (16 rows: one, which keeps the registers
// for the weights: a whole pass takes 18.1 us against 17.6 at 16 rows, N 4096, K 14336,
// groups of 32, and 86 against 82 for 48 tokens, top 8 of 64 experts, N 4096, K 2048).
BSR_HD constexpr uint32_t w4g_stage(uint32_t rows, uint32_t ct, uint32_t gpc) {
    return rows <= kW4gFew ? w4g_pass(ct, gpc) : 1;
}
// LDS bytes of one staged row (16 of padding spread the 16 rows read at one
// offset over the banks).
BSR_HD constexpr uint32_t w4g_pitch(uint32_t stage) { return stage * kW4gChunk * 2 + 16; }
// Waves per workgroup: 16 leave a wave 128 registers, which the kernels of one
// column tile and few rows fit.
BSR_HD constexpr uint32_t w4g_max_waves(uint32_t rows, uint32_t ct) { return rows <= kW4gFew && ct == 1 ? 16 : 8; }
static_assert(w4g_max_waves(kW4gFew, 1) * kW4gFew * w4g_pitch(w4g_stage(kW4gFew, 1, 0)) <= kLdsBytes &&
                  w4g_max_waves(kW4gFew, 2) * kW4gFew * w4g_pitch(w4g_stage(kW4gFew, 2, 0)) <= kLdsBytes &&
                  w4g_max_waves(kW4gRows, 1) * kW4gRows * w4g_pitch(w4g_stage(kW4gRows, 1, 0)) <= kLdsBytes,
              "what the waves of a workgroup stage fits, and so do their sums (1 KB a wave and column tile)");

struct W4gPlan {
    uint32_t rows;  // of a tile, at most: kW4gFew or kW4gRows
    uint32_t ct;    // column tiles per workgroup (with the SiLU product: a gate and an up tile)
    uint32_t row_tiles, col_tiles, waves, chunks_per_wave, wave_bytes, lds;
};

inline W4gPlan w4_group_plan(uint32_t rows, uint32_t experts, uint32_t cols, uint32_t k, uint32_t group, bool silu) {
    W4gPlan p;
    const uint32_t gpc = group == 0 ? 0 : kW4gChunk / group;
    const uint32_t used = rows < experts ? rows : experts;
    // Tiles of 4 rows where an expert has 2 on average: a token's few rows, and
    // less to stage; the experts with more read their weight again from cache
    // (16 tokens, top 8 of 64 experts, with the SiLU product 65-70 us, with tiles of 16 73).
    p.rows = rows <= kW4gFew || rows <= 2 * (uint64_t)used ? kW4gFew : kW4gRows;
    const uint32_t chunks = (uint32_t)div_up(k, kW4gChunk);
    p.row_tiles = (uint32_t)grouped_row_tiles(rows, experts, p.rows);
    // Two column tiles share the staged activations from 5 rows on, if that
    // leaves every CU a workgroup (48 tokens, top 8 of 64 experts, N 4096, K 2048: 82 us
    // against 97; at 256 tiles of 16 columns one tile each is faster, 17.6 against 23.3).
    const uint64_t tiles = (uint64_t)p.row_tiles * div_up(cols, kW4gCols);
    p.ct = silu || (p.rows > kW4gFew && tiles >= 2 * (uint64_t)kGemmCus) ? 2 : 1;
    p.col_tiles = (uint32_t)div_up(cols, kW4gCols * (silu ? 1 : p.ct));
    // As many waves as run at once (16, 12 or 8 per CU by their registers), so
    // that one round of workgroups takes the whole weight.
    const uint32_t at_once = (p.rows > kW4gFew ? 8 : (p.ct == 2 ? 12 : 16)) * kGemmCus;
    const uint32_t most = w4g_max_waves(p.rows, p.ct), pass = w4g_pass(p.ct, gpc);
    uint64_t waves = at_once / ((uint64_t)p.row_tiles * p.col_tiles);
    waves = waves > 1 ? waves : 1;
    waves = waves < most ? waves : most;
    waves = waves < chunks ? waves : chunks;
    p.chunks_per_wave = (uint32_t)div_up(div_up(chunks, waves), pass) * pass;  // whole passes
    p.waves = (uint32_t)div_up(chunks, p.chunks_per_wave);
    p.wave_bytes = (rows < p.rows ? rows : p.rows) * w4g_pitch(w4g_stage(p.rows, p.ct, gpc));
    const uint32_t sums = p.waves * 64 * 4 * 4 * p.ct;
    p.lds = p.waves * p.wave_bytes;
    p.lds = p.lds > sums ? p.lds : sums;
    return p;
}

inline uint64_t w4_group_threads(const W4gPlan &p) { return (uint64_t)p.row_tiles * p.col_tiles * p.waves * 64; }

}  // namespace bsr
