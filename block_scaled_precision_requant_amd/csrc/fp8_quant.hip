// fp8_quant.hip -- BF16 weight to E4M3 codes with one scale per block of 128 x 128,
// and the transposed codes beside them.
//
// s = fl32(amax / 448) over the block, code = the E4M3 value nearest fl32(v / s).  A
// workgroup owns one block: a lane holds 8 rows by 8 columns of it in registers, so
// the block is read once for its maximum and its codes.  A square block has the same
// scale in the transposed weight: each lane turns its 8 x 8 codes with byte permutes
// and the workgroup turns the 16 x 16 lanes through LDS, so that the transposed rows
// leave as whole 128-byte lines too.  Bound by HBM: 3 bytes an element, 4 with the
// transposed codes.  MI355X, 8 weights of 4096 x 4096 with the transposed codes (537
// MB): 105 us, 5.1 TB/s, as a device copy of 1 GiB reaches; vector issue, for the
// divisions and conversions, is at 65 % beside it.  One of 1000 x 2048 takes 6.2.
#include "fp8_internal.h"

namespace bsr {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// E4M3 codes of four quotients, clamped to the largest value (v_cvt_pk_fp8_f32
// rounds to nearest, ties to even, subnormals included).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    auto cut = [](float x) { return fminf(fmaxf(x, -448.0f), 448.0f); };
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(cut(a), cut(b), 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cut(c), cut(d), lo, true);
}

// 4 x 4 bytes transposed: byte j of out[i] = byte i of in[j].
__device__ __forceinline__ void turn4(uint32_t (&x)[4]) {
    const uint32_t a = __builtin_amdgcn_perm(x[1], x[0], 0x05010400), b = __builtin_amdgcn_perm(x[3], x[2], 0x05010400);
    const uint32_t c = __builtin_amdgcn_perm(x[1], x[0], 0x07030602), d = __builtin_amdgcn_perm(x[3], x[2], 0x07030602);
    x[0] = __builtin_amdgcn_perm(b, a, 0x05040100);
    x[1] = __builtin_amdgcn_perm(b, a, 0x07060302);
    x[2] = __builtin_amdgcn_perm(d, c, 0x05040100);
    x[3] = __builtin_amdgcn_perm(d, c, 0x07060302);
}

template <bool TURN>
__global__ __launch_bounds__(kQwThreads) void quantize_w_fp8_kernel(const uint16_t *__restrict__ w, uint8_t *__restrict__ q,
                                                                    float *__restrict__ scale, uint8_t *__restrict__ qt,
                                                                    float *__restrict__ scale_t, uint32_t n, uint32_t k) {
    __shared__ uint32_t peak[kQwThreads / 64];
    __shared__ __attribute__((aligned(16))) uint8_t turned[TURN ? kFp8Block * kFp8Block : 16];
    const uint32_t nb = k / kFp8Block, blocks = (n + kFp8Block - 1) / kFp8Block;
    const uint32_t kb = blockIdx.x % nb, rb = blockIdx.x / nb % blocks;
    const uint64_t e = blockIdx.x / nb / blocks;
    const uint32_t tid = threadIdx.x, col = tid % 16, group = tid / 16;  // 8 columns and 8 rows of the block
    const uint64_t row0 = e * n + rb * kFp8Block + group * 8;
    const uint32_t live = n - rb * kFp8Block;  // rows of the block inside the weight, if below 128
    const uint64_t at = row0 * k + kb * kFp8Block + col * 8;

    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = group * 8 + i < live ? *reinterpret_cast<const u32x4 *>(w + at + (uint64_t)i * k) : u32x4{0, 0, 0, 0};
    // a BF16's magnitude orders as its bits do
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) most = max(most, max(v[i][j] & 0x7FFFu, v[i][j] >> 16 & 0x7FFFu));
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, d));
    if (tid % 64 == 0) peak[tid / 64] = most;
    __syncthreads();
#pragma unroll
    for (uint32_t i = 0; i < kQwThreads / 64; ++i) most = max(most, peak[i]);
    const float s = __uint_as_float(most << 16) / 448.0f;
    if (tid == 0) {
        scale[(e * blocks + rb) * nb + kb] = s;
        if constexpr (TURN) scale_t[(e * nb + kb) * blocks + rb] = s;
    }
    uint32_t code[8][2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t pair = v[i][2 * h + j / 2];
                x[j] = s > 0.0f ? __uint_as_float(j % 2 ? pair & 0xFFFF0000u : pair << 16) / s : 0.0f;
            }
            code[i][h] = e4m3x4(x[0], x[1], x[2], x[3]);
        }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (group * 8 + i < live)
            *reinterpret_cast<uint2 *>(q + at + (uint64_t)i * k) = make_uint2(code[i][0], code[i][1]);
    if constexpr (TURN) {  // (n is a multiple of 128: every row of the block is live)
        // LDS rows are the 128 columns; the 8 bytes of row group g of a column of lane
        // column c sit at slot g ^ c, so that 16 lanes write 16 slots
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t a[4] = {code[0][h], code[1][h], code[2][h], code[3][h]};
            uint32_t b[4] = {code[4][h], code[5][h], code[6][h], code[7][h]};
            turn4(a);
            turn4(b);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint2 *>(turned + (col * 8 + h * 4 + j) * kFp8Block + (group ^ col) * 8) =
                    make_uint2(a[j], b[j]);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t r = i * 32 + tid / 8, u = tid % 8, x = r / 8;  // column of the block, 16 bytes of it
            u32x4 o = *reinterpret_cast<const u32x4 *>(turned + r * kFp8Block + ((2 * u ^ x) & ~1u) * 8);
            if (x & 1) o = u32x4{o[2], o[3], o[0], o[1]};
            *reinterpret_cast<u32x4 *>(qt + ((e * nb + kb) * kFp8Block + r) * n + rb * kFp8Block + u * 16) = o;
        }
    }
}

}  // namespace

hipError_t launch_quantize_w_fp8(const uint16_t *w, uint8_t *q, float *scale, uint8_t *qt, float *scale_t,
                                 uint32_t experts, uint32_t n, uint32_t k, hipStream_t s) {
    const uint32_t grid = (uint32_t)(experts * div_up(n, kFp8Block) * (k / kFp8Block));
    auto kernel = qt != nullptr ? quantize_w_fp8_kernel<true> : quantize_w_fp8_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kQwThreads), 0, s, w, q, scale, qt, scale_t, n, k);
    return hipGetLastError();
}

}  // namespace bsr
