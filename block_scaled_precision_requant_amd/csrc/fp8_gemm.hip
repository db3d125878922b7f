// fp8_gemm.hip -- the FP8 products: which kernel a call runs (fp8_choice).
#include "fp8_internal.h"

namespace bsr {

hipError_t launch_fp8_gemm(const Fp8Args &p, hipStream_t s) {
    const Fp8Choice c = fp8_choice(p.rows.rows, p.rows.experts, p.n, p.k, p.silu);
    if (c.stream) return launch_fp8_stream(p, c.plan, s);
    const uint32_t bm = fp8_shape(c.shape).bm;
    if (bm <= 32) return launch_fp8_tiles_few(p, c, s);
    if (bm <= 64) return launch_fp8_tiles_64(p, c, s);
    return bm <= 128 ? launch_fp8_tiles_128(p, c, s) : launch_fp8_tiles_256(p, c, s);
}

}  // namespace bsr
