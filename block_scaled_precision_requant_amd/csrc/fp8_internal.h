// fp8_internal.h -- launchers and device helpers of the FP8 products, the weight
// quantizer and the kernels around sorted tokens.
#pragma once

#include "fp8_geometry.h"
#include "moe_internal.h"

namespace bsr {

// Operands of an FP8 product (no validation: the C-ABI layer has checked every
// argument).  offsets null in `rows`: dense, one weight for all rows.
struct Fp8Args {
    const uint8_t *a, *w;
    const float *a_s, *w_s;
    uint16_t *out;
    GroupedRows rows;
    uint32_t n, k;
    bool silu;
};

hipError_t launch_fp8_gemm(const Fp8Args &p, hipStream_t s);
hipError_t launch_fp8_stream(const Fp8Args &p, const Fp8StreamPlan &plan, hipStream_t s);
hipError_t launch_fp8_tiles_few(const Fp8Args &p, const Fp8Choice &c, hipStream_t s);
hipError_t launch_fp8_tiles_64(const Fp8Args &p, const Fp8Choice &c, hipStream_t s);
hipError_t launch_fp8_tiles_128(const Fp8Args &p, const Fp8Choice &c, hipStream_t s);
hipError_t launch_fp8_tiles_256(const Fp8Args &p, const Fp8Choice &c, hipStream_t s);
hipError_t launch_quantize_w_fp8(const uint16_t *w, uint8_t *q, float *scale, uint8_t *qt, float *scale_t,
                                 uint32_t experts, uint32_t n, uint32_t k, hipStream_t s);
hipError_t launch_moe_dispatch(const uint16_t *x, const int32_t *pos, uint16_t *out, uint32_t tokens, uint32_t top_k,
                               uint32_t rows, uint32_t n, hipStream_t s);
hipError_t launch_moe_dispatch_grad(const uint16_t *d_rows, const int32_t *pos, uint16_t *d_x, uint32_t tokens,
                                    uint32_t top_k, uint32_t rows, uint32_t n, hipStream_t s);
hipError_t launch_moe_combine_grad(const uint16_t *d_out, const uint16_t *y, const int32_t *pos, const float *weights,
                                   uint16_t *d_y, float *d_weights, uint32_t tokens, uint32_t top_k, uint32_t rows,
                                   uint32_t n, hipStream_t s);

#ifdef __HIPCC__
typedef int v8i __attribute__((ext_vector_type(8)));

// BF16 nearest to x, ties to even, and NaN for NaN (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint16_t f32_to_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ uint2 f32_to_bf16x4(v4f v) {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(uint2, __builtin_convertvector(v, b4));
}

// Sixteen rows of E4M3 codes times sixteen others over one block of 128: lane l holds
// 32 codes of row l % 16 of `w` and of `a`, the same elements of the block for both;
// its result is out(a row l % 16, w row 4 * (l / 16) + r), in binary32.  (Scale
// operands of 0 select the instruction without block exponents.)
__device__ __forceinline__ v4f fp8_dot16(v8i w, v8i a) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}

// gate / (1 + exp(-gate)) * up; for gate below -88.7 the quotient is -0.  exp(-gate) as the
// hardware's 2^t and the quotient by its reciprocal, each good to one step of binary32; t is
// rounded, which for a negative gate moves the result by up to 1.25 |gate| 2^-24, below
// 2^-17 where it is not 0 (BF16 rounds at 2^-8).  The reciprocal is of a quarter, so that it
// is normal for every finite exp(-gate); its own quarter is 2^-22 off at most where that is
// subnormal (gate below -87.3, where the bound has 2^-19 to spare), while a quarter of the gate
// would cut a subnormal gate's bits.  (8192 rows over 8 uneven experts, n 28672, k 4096, in
// one comparison: 934 us, with expf and a division 982, the epilogue being a tenth of a tile's time.)
__device__ __forceinline__ float silu_product(float gate, float up) {
    const float e = __builtin_amdgcn_exp2f(gate * -1.44269504f);
    return gate * (__builtin_amdgcn_rcpf(fmaf(e, 0.25f, 0.25f)) * 0.25f) * up;
}

// Eight elements of a row of n, from c on; rows of any alignment (one 16-byte access at
// any even address where all eight are there, else element by element).
typedef uint16_t u16x8 __attribute__((ext_vector_type(8), aligned(2)));

__device__ __forceinline__ u16x8 load8(const uint16_t *p, uint32_t c, uint32_t n) {
    if (c + 8 <= n) return *reinterpret_cast<const u16x8 *>(p + c);
    u16x8 v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (c + i < n) v[i] = p[c + i];
    return v;
}
__device__ __forceinline__ void store8(uint16_t *p, uint32_t c, uint32_t n, u16x8 v) {
    if (c + 8 <= n) {
        *reinterpret_cast<u16x8 *>(p + c) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (c + i < n) p[c + i] = v[i];
}

// Four columns of one output row, those below n.  `wide`: out and n keep 8-byte words whole.
__device__ __forceinline__ void store4(uint16_t *out, uint64_t row, uint32_t col, uint32_t n, v4f v, bool wide) {
    uint16_t *p = out + row * n + col;
    if (wide) {
        if (col < n)
            *reinterpret_cast<uint2 *>(p) = f32_to_bf16x4(v);
        return;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (col + r < n) p[r] = f32_to_bf16(v[r]);
}
#endif

}  // namespace bsr
