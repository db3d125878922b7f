// grouped.hip -- int8 block-scaled products grouped by expert.
//
// out[p, j] = bf16_rne( sum_b fl32(a_s[i,b] * w_s[e,j,b]) * P[i,e,j,b] ): the
// result of the GEMM in gemm.hip, with the weight of row p's expert e and
// operand row i = row_index[p] (the grouped W8A8 expert product of page
// "metrale_model_layers/layers/ops/fp8_moe_grouped_tc_w8a8.rs").
//
// The offsets are device values, so the host launches as many workgroups as
// any offsets could need and each finds its tile itself: a lane per expert
// counts row tiles, wave prefixes give their totals and the tile of this
// workgroup; workgroups past the total leave.  The tiles are those of
// gemm_tile.h, their A rows gathered through row_index by the staging itself,
// so no gathered copy of the activations is made.  Few rows per expert run in
// grouped_gemv.hip instead (grouped_gemv_rule).
#include "gemm_tile.h"
#include "moe_internal.h"

namespace bsr {
namespace gemm_kernels {

// One tile of up to 128 x 128 outputs, four waves of 64 x 64, two workgroups
// per CU.  An expert's last rows, when 96, 64 or 32 hold them, take a wave grid
// that computes no more than that: each of the four waves 96 x 32, 64 x 32 or
// 32 x 32.  MI355X: 8192 rows over 8 experts, n 28672, k 4096, 2.49-2.54 ms (757-772
// TOPS; the dense GEMM of that size 844), bound by the FP32 rescale of each block
// as the dense GEMM is; 6016 rows over 32 uneven experts, n 4096, k 2048, 176-198 us by
// their routing (510-574 TOPS), where the rest goes to the experts' remainders: tiles that
// are part empty, stage their scales four blocks at a time and hold 32 columns a wave.
template <bool GATHER>
__global__ __launch_bounds__(256, 2) void grouped_kernel(
    const int8_t *__restrict__ a, const int8_t *__restrict__ w, const float *__restrict__ a_s,
    const float *__restrict__ w_s, uint16_t *__restrict__ out, GroupedRows g, uint32_t N, uint32_t K,
    uint32_t tiles_n) {
    constexpr int BM = kGemmBM, BN = kGemmBN;
    constexpr size_t kLds = TileTraits<BM, BN, 64, 64, 1, 2, false>::kLds;
    static_assert(TileTraits<96, BN, 96, 32, 1, 2, false>::kLds <= kLds, "the smaller tiles fit");
    __shared__ __attribute__((aligned(1024))) char lds[kLds];
    ClassedTiles<kGemmBM> rt(g, threadIdx.x & 63);
    // (overlapping ranges could ask for more tiles than the grid has: those are not computed)
    const uint32_t tiles_m = min(rt.n0 + rt.n1 + rt.n2, gridDim.x / tiles_n);
    if (blockIdx.x >= tiles_m * tiles_n) return;
    uint32_t tm, tn;
    grouped_tile_of<kGemmGroupM>(blockIdx.x, tiles_m, tiles_n, tm, tn);
    RowTile r = rt.find(tm);
    // the same in every lane; said so, since a buffer descriptor that the compiler
    // takes for a vector costs a loop around each copy
    r.expert = __builtin_amdgcn_readfirstlane(r.expert);
    r.row0 = __builtin_amdgcn_readfirstlane(r.row0);
    r.rows = __builtin_amdgcn_readfirstlane(r.rows);
    if (r.rows == 0) return;
    const uint32_t n0 = __builtin_amdgcn_readfirstlane(tn * BN), nb = K / 32;
    const uint64_t wrow = (uint64_t)r.expert * N + n0;
    TileArgs t = {a, w + wrow * K, a_s, w_s + wrow * nb, nullptr, r.rows, min((uint32_t)BN, N - n0), 0,
                  r.row0, n0, r.row0 + r.rows};
    if constexpr (GATHER) {
        t.index = g.index + r.row0;
        t.buf_rows = __builtin_amdgcn_readfirstlane(g.src_rows);
    } else {
        t.a += (uint64_t)r.row0 * K;
        t.a_s += (uint64_t)r.row0 * nb;
        t.buf_rows = r.rows;
    }
    if (r.rows <= 32)
        gemm_tile<32, BN, 32, 32, 1, 2, false, GATHER>(lds, t, out, N, K, nb, 0, nullptr, 0, 0, 0);
    else if (r.rows <= 64)
        gemm_tile<64, BN, 64, 32, 1, 2, false, GATHER>(lds, t, out, N, K, nb, 0, nullptr, 0, 0, 0);
    else if (r.rows <= 96)
        gemm_tile<96, BN, 96, 32, 1, 2, false, GATHER>(lds, t, out, N, K, nb, 0, nullptr, 0, 0, 0);
    else
        gemm_tile<BM, BN, 64, 64, 1, 2, false, GATHER>(lds, t, out, N, K, nb, 0, nullptr, 0, 0, 0);
}

}  // namespace gemm_kernels

hipError_t launch_grouped_gemm(const int8_t *a, const int8_t *w, const float *a_s, const float *w_s, uint16_t *out,
                               const GroupedRows &g, uint32_t n, uint32_t k, hipStream_t s) {
    if (grouped_gemv_rule(g.rows, g.experts, n))
        return launch_grouped_gemv(a, w, a_s, w_s, out, g, n, k, grouped_gemv_plan(g.rows, g.experts, n, k), s);
    const uint32_t tiles_n = (uint32_t)div_up(n, kGemmBN);
    const uint64_t grid = grouped_row_tiles(g.rows, g.experts, kGemmBM) * tiles_n;
    auto kernel = g.index != nullptr ? gemm_kernels::grouped_kernel<true> : gemm_kernels::grouped_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(256), 0, s, a, w, a_s, w_s, out, g, n, k, tiles_n);
    return hipGetLastError();
}

}  // namespace bsr
