// Instances of the FP8 tile kernel whose assembly test_fp8_copies.py looks at.
#include "fp8_tile.h"

namespace bsr::fp8_kernels {

#define BSR_KERNEL(...)                                                                                            \
    template __global__ void fp8_gemm_kernel<__VA_ARGS__>(const uint8_t *, const uint8_t *, const float *, const float *, \
                                                          uint16_t *, GroupedRows, uint32_t, uint32_t, uint32_t, uint32_t)
// one row of matrix products a wave: the dense shapes of 16 rows
BSR_KERNEL(16, 16, 16, 16, 4, 4, false, kDense);
BSR_KERNEL(16, 32, 16, 32, 4, 4, false, kDense);
BSR_KERNEL(16, 64, 16, 64, 3, 4, false, kDense);
BSR_KERNEL(16, 128, 16, 128, 2, 4, false, kDense);
// ... and last rows of an expert, at half and at a quarter of the height
BSR_KERNEL(64, 128, 32, 64, 3, 1, false, kGrouped);
BSR_KERNEL(128, 128, 64, 64, 2, 1, true, kGathered);
// two and more
BSR_KERNEL(32, 16, 32, 16, 4, 4, false, kDense);
BSR_KERNEL(64, 64, 64, 32, 3, 2, false, kDense);
BSR_KERNEL(256, 256, 128, 64, 2, 1, false, kDense);

}  // namespace bsr::fp8_kernels
