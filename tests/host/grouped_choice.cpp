// Prints which kernel a grouped product of (rows, experts, n) takes: "gemv R" with R rows a tile, or "tiles".
#include <cstdio>
#include <cstdlib>

#include "moe_geometry.h"

int main(int argc, char **argv) {
    if (argc != 5) return 2;
    uint32_t v[4];
    for (int i = 0; i < 4; ++i) v[i] = (uint32_t)std::strtoul(argv[i + 1], nullptr, 10);
    if (bsr::grouped_gemv_rule(v[0], v[1], v[2]))
        std::printf("gemv %u\n", bsr::grouped_gemv_plan(v[0], v[1], v[2], v[3]).rows);
    else
        std::printf("tiles\n");
    return 0;
}
