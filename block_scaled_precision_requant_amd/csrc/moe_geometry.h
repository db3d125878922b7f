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

}  // namespace bsr
