// grouped.hip -- int8 block-scaled products grouped by expert.
//
// out[p, j] = bf16_rne( sum_b fl32(a_s[i,b] * w_s[e,j,b]) * P[i,e,j,b] ): the
// result of the GEMM in gemm.hip, with the weight of row p's expert e and
// operand row i = row_index[p] (the grouped W8A8 expert product of page
// "metrale_model_layers/layers/ops/fp8_moe_grouped_tc_w8a8.rs").
//
// A workgroup takes 16 rows of one expert and 64 columns, a wave 16 of them;
// per 32-wide block one v_mfma_i32_16x16x32_i8 gives the exact P.
#include "moe_internal.h"

namespace bsr {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr uint32_t kRows = 16, kCols = 64;

__global__ __launch_bounds__(256) void grouped_gemm_kernel(const int8_t *__restrict__ a, const int8_t *__restrict__ w,
                                                           const float *__restrict__ a_s,
                                                           const float *__restrict__ w_s, uint16_t *__restrict__ out,
                                                           GroupedRows g, uint32_t n, uint32_t k, uint32_t col_tiles) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const RowTile t = find_row_tile(g, kRows, blockIdx.x / col_tiles, lane);
    if (t.rows == 0) return;
    const uint32_t c = lane & 15, q = lane >> 4;
    const uint32_t col = (blockIdx.x % col_tiles) * kCols + wave * 16 + c;
    const uint32_t nb = k / 32;
    const uint64_t wrow = (uint64_t)t.expert * n + min(col, n - 1);
    const int32_t src = c < t.rows ? source_row(g, t.row0 + c) : -1;
    const int8_t *wp = w + wrow * k + 8 * q;
    const float *wsp = w_s + wrow * nb;
    const int8_t *ap = a + (uint64_t)max(src, 0) * k + 8 * q;
    int32_t srow[4];  // this lane's output rows 4 q + r
#pragma unroll
    for (int r = 0; r < 4; ++r) srow[r] = 4 * q + r < t.rows ? source_row(g, t.row0 + 4 * q + r) : -1;
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (uint32_t b = 0; b < nb; ++b) {
        const long av = *reinterpret_cast<const long *>(ap + 32 * (uint64_t)b);
        const long wv = *reinterpret_cast<const long *>(wp + 32 * (uint64_t)b);
        const v4i p = __builtin_amdgcn_mfma_i32_16x16x32_i8(src < 0 ? 0 : av, wv, v4i{0, 0, 0, 0}, 0, 0, 0);
        const float ws = wsp[b];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float as = srow[r] < 0 ? 0.0f : a_s[(uint64_t)srow[r] * nb + b];
            acc[r] = fmaf((float)p[r], as * ws, acc[r]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * q + r < t.rows && col < n) out[(uint64_t)(t.row0 + 4 * q + r) * n + col] = f32_to_bf16_rne(acc[r]);
}

}  // namespace

hipError_t launch_grouped_gemm(const int8_t *a, const int8_t *w, const float *a_s, const float *w_s, uint16_t *out,
                               const GroupedRows &g, uint32_t n, uint32_t k, hipStream_t s) {
    const uint32_t col_tiles = (uint32_t)div_up(n, kCols);
    const uint64_t grid = grouped_row_tiles(g.rows, g.experts, kRows) * col_tiles;
    hipLaunchKernelGGL(grouped_gemm_kernel, dim3((uint32_t)grid), dim3(256), 0, s, a, w, a_s, w_s, out, g, n, k,
                       col_tiles);
    return hipGetLastError();
}

}  // namespace bsr
