// Prints which kernel fp8_choice takes: "rows experts n k silu" a line on stdin,
// "shape bm bn tiles_m tiles_n threads" (shape -1: streamed) a line on stdout.
#include <cstdio>

#include "fp8_geometry.h"

int main() {
    unsigned rows, experts, n, k, silu;
    while (std::scanf("%u %u %u %u %u", &rows, &experts, &n, &k, &silu) == 5) {
        const bsr::Fp8Choice c = bsr::fp8_choice(rows, experts, n, k, silu != 0);
        if (c.stream)
            std::printf("-1 16 16 %u %u %llu\n", c.plan.row_tiles, c.plan.col_tiles, (unsigned long long)c.threads);
        else
            std::printf("%u %u %u %u %u %llu\n", c.shape, bsr::fp8_shape(c.shape).bm, bsr::fp8_shape(c.shape).bn, c.tiles_m,
                        c.tiles_n, (unsigned long long)c.threads);
    }
}
