// fp8_tiles_128.hip -- FP8 product tiles of 128 rows.
#include "fp8_tile.h"

namespace bsr {

hipError_t launch_fp8_tiles_128(const Fp8Args &p, const Fp8Choice &c, hipStream_t s) {
    using namespace fp8_kernels;
    switch (c.shape) {
    case 12: launch_tile<12, 64, 32, 3, 2>(p, c, s); break;
    case 13: launch_tile<13, 64, 32, 4, 1>(p, c, s); break;
    case kFp8PairIndex: launch_tile<kFp8PairIndex, 64, 64, 2, 1>(p, c, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace bsr
