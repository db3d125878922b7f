// fp8_tiles_64.hip -- FP8 product tiles of 64 rows.
#include "fp8_tile.h"

namespace bsr {

hipError_t launch_fp8_tiles_64(const Fp8Args &p, const Fp8Choice &c, hipStream_t s) {
    using namespace fp8_kernels;
    switch (c.shape) {
    case 8: launch_tile<8, 64, 16, 3, 4>(p, c, s); break;
    case 9: launch_tile<9, 64, 32, 3, 4>(p, c, s); break;
    case 10: launch_tile<10, 64, 32, 3, 2>(p, c, s); break;
    case 11: launch_tile<11, 32, 64, 3, 1>(p, c, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace bsr
