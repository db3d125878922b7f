// fp8_tiles_few.hip -- FP8 product tiles of 16 and 32 rows: the waves split K, each with a
// ring of its own, and meet only to add their sums.
#include "fp8_tile.h"

namespace bsr {

hipError_t launch_fp8_tiles_few(const Fp8Args &p, const Fp8Choice &c, hipStream_t s) {
    using namespace fp8_kernels;
    switch (c.shape) {
    case 0: launch_tile<0, 16, 16, 4, 4>(p, c, s); break;
    case 1: launch_tile<1, 16, 32, 4, 4>(p, c, s); break;
    case 2: launch_tile<2, 16, 64, 3, 4>(p, c, s); break;
    case 3: launch_tile<3, 16, 128, 2, 4>(p, c, s); break;
    case 4: launch_tile<4, 32, 16, 4, 4>(p, c, s); break;
    case 5: launch_tile<5, 32, 32, 3, 4>(p, c, s); break;
    case 6: launch_tile<6, 32, 64, 3, 4>(p, c, s); break;
    case 7: launch_tile<7, 32, 128, 2, 3>(p, c, s); break;
    default: return hipErrorInvalidValue;
    }
    return hipGetLastError();
}

}  // namespace bsr
