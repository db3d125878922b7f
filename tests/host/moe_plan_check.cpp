// Host check of the expert-layer launch plans (the code the launchers run):
// every chunk of K belongs to one wave, no wave is without one, LDS and
// workgroup sizes stay in their bounds, the row-tile bound covers any offsets,
// and the router's workspace stays within 1024 bytes per expert.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "moe_geometry.h"

using namespace bsr;

static void fail(const char *what, uint64_t a, uint64_t b, uint64_t c, uint64_t d) {
    std::printf("%s at %llu %llu %llu %llu\n", what, (unsigned long long)a, (unsigned long long)b, (unsigned long long)c,
                (unsigned long long)d);
    std::exit(1);
}

int main() {
    uint64_t cases = 0, many = 0, gemv = 0;
    const uint32_t rows[] = {1, 2, 3, 4, 5, 8, 15, 16, 17, 48, 64, 384, 1000, 6000, 32768};
    const uint32_t experts[] = {1, 2, 7, 8, 64, 65, 128, 1000};
    const uint32_t ns[] = {1, 15, 16, 17, 100, 512, 1000, 4096, 14336, 28672};
    const uint32_t ks[] = {32, 64, 96, 128, 160, 256, 1056, 2048, 4096, 4128, 14336, 131072};
    for (uint32_t r : rows)
        for (uint32_t e : experts)
            for (uint32_t n : ns)
                for (uint32_t k : ks) {
                    for (uint32_t group : {0u, 32u, 64u, 128u})
                        for (int silu = 0; silu < 2; ++silu) {
                            if (group != 0 && k % group != 0) continue;
                            const W4gPlan p = w4_group_plan(r, e, n, k, group, silu != 0);
                            const uint32_t gpc = group == 0 ? 0 : kW4gChunk / group;
                            const uint64_t chunks = div_up(k, kW4gChunk);
                            if (p.waves < 1 || p.waves > w4g_max_waves(p.rows, p.ct)) fail("waves", r, e, n, k);
                            if ((uint64_t)p.waves * p.chunks_per_wave < chunks) fail("K not covered", r, e, n, k);
                            if ((uint64_t)(p.waves - 1) * p.chunks_per_wave >= chunks) fail("idle wave", r, e, n, k);
                            if (p.chunks_per_wave % w4g_pass(p.ct, gpc) != 0) fail("part of a pass", r, e, n, k);
                            if (p.lds > kLdsBytes || p.lds < p.waves * 1024 * p.ct) fail("lds", r, e, n, k);
                            const uint32_t most = r < p.rows ? r : p.rows;
                            if (p.wave_bytes < most * w4g_pitch(w4g_stage(p.rows, p.ct, gpc))) fail("stage", r, e, n, k);
                            if (p.row_tiles != grouped_row_tiles(r, e, p.rows)) fail("row tiles", r, e, n, k);
                            if ((uint64_t)p.col_tiles * kW4gCols * (silu ? 1 : p.ct) < n) fail("columns", r, e, n, k);
                            ++cases;
                            many += p.rows == kW4gRows;
                        }
                    const GroupedGemvPlan g = grouped_gemv_plan(r, e, n, k);
                    const uint64_t chunks = div_up(k, kGgChunk);
                    if (g.waves < 1 || g.waves > gg_max_waves(g.rows)) fail("gemv waves", r, e, n, k);
                    if ((uint64_t)g.waves * g.chunks_per_wave < chunks) fail("gemv K not covered", r, e, n, k);
                    if ((uint64_t)(g.waves - 1) * g.chunks_per_wave >= chunks) fail("gemv idle wave", r, e, n, k);
                    if (g.lds > kLdsBytes || g.lds < g.waves * gg_wave_bytes(g.rows) || g.lds < g.waves * 1024)
                        fail("gemv lds", r, e, n, k);
                    gemv += grouped_gemv_rule(r, e, n);
                    ++cases;
                }
    // the bound on row tiles against the worst offsets: one row each, the rest in one
    for (uint32_t r : rows)
        for (uint32_t e : experts)
            for (uint32_t bm : {4u, 16u, 128u}) {
                const uint64_t bound = grouped_row_tiles(r, e, bm);
                std::vector<uint64_t> c(e, 0);
                uint64_t left = r;
                for (uint32_t i = 0; i + 1 < e && left > 1; ++i) {
                    c[i] = 1;
                    --left;
                }
                c[e - 1] = left;
                uint64_t tiles = 0;
                for (uint64_t x : c) tiles += div_up(x, bm);
                if (tiles > bound) fail("tile bound", r, e, bm, tiles);
                uint64_t even = 0;
                for (uint32_t i = 0; i < e; ++i) even += div_up(r / e + (i < r % e), bm);
                if (even > bound) fail("even tile bound", r, e, bm, even);
                ++cases;
            }
    for (uint32_t e = 1; e <= kRouteMaxExperts; ++e)
        for (uint64_t t = 0; t < (1ull << 31); t = t * 3 + 1) {
            const RoutePlan p = moe_route_plan((uint32_t)t, e);
            if (p.bytes > 1024ull * e || p.blocks > kRouteMaxBlocks) fail("route workspace", t, e, p.blocks, p.bytes);
            if ((uint64_t)p.blocks * p.per_block < t) fail("tokens not covered", t, e, p.blocks, p.per_block);
            if (p.blocks > 1 && (uint64_t)(p.blocks - 1) * p.per_block >= t) fail("empty run", t, e, p.blocks, p.per_block);
            if ((p.blocks <= 1) != (p.bytes == 0)) fail("workspace of one run", t, e, p.blocks, p.bytes);
            ++cases;
        }
    std::printf("ok %llu %llu %llu\n", (unsigned long long)cases, (unsigned long long)many, (unsigned long long)gemv);
    return 0;
}
