// fp8_tiles_256.hip -- FP8 product tiles of 256 rows.
#include "fp8_tile.h"

namespace bsr {

hipError_t launch_fp8_tiles_256(const Fp8Args &p, const Fp8Choice &c, hipStream_t s) {
    using namespace fp8_kernels;
    switch (c.shape) {
    case 14: launch_tile<14, 128, 32, 3, 1>(p, c, s); break;
    case 15: launch_tile<15, 128, 64, 2, 1>(p, c, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace bsr
