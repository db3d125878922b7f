// grouped.hip -- int8 block-scaled products grouped by expert.
//
// out[p, j] = bf16_rne( sum_b fl32(a_s[i,b] * w_s[e,j,b]) * P[i,e,j,b] ): the
// result of the GEMM in gemm.hip, with the weight of row p's expert e and
// operand row i = row_index[p] (the grouped W8A8 expert product of page
// "metrale_model_layers/layers/ops/fp8_moe_grouped_tc_w8a8.rs").
//
// The offsets are device values, so the host launches as many workgroups as
// any offsets could need and each finds its tile itself: a lane per expert
// counts row tiles, a wave prefix gives their total and the tile of this
// workgroup; workgroups past the total leave.  The tiles are those of
// gemm_tile.h, their A rows gathered through row_index by the staging itself,
// so no gathered copy of the activations is made.
#include "gemm_tile.h"
#include "moe_internal.h"

namespace bsr {
namespace gemm_kernels {

template <int BM, int BN, int WM, int WN, int WG_PER_CU, int RING, bool GATHER>
__global__ __launch_bounds__(BM * BN / (WM * WN) * 64, WG_PER_CU) void grouped_kernel(
    const int8_t *__restrict__ a, const int8_t *__restrict__ w, const float *__restrict__ a_s,
    const float *__restrict__ w_s, uint16_t *__restrict__ out, GroupedRows g, uint32_t N, uint32_t K,
    uint32_t tiles_n) {
    RowTiles rt(g, BM, threadIdx.x & 63);
    const uint64_t tiles_m = rt.count();
    if (blockIdx.x >= tiles_m * tiles_n) return;
    uint32_t tm, tn;
    tile_of<BM == kGemmTallBM ? kGemmTallGroupM : kGemmGroupM>(
        blockIdx.x, (uint32_t)min(tiles_m, (uint64_t)(gridDim.x / tiles_n)), tiles_n, tm, tn);
    const RowTile r = rt.find(tm);
    if (r.rows == 0) return;
    const uint32_t n0 = tn * BN, nb = K / 32;
    const uint64_t wrow = (uint64_t)r.expert * N + n0;
    TileArgs t = {a, w + wrow * K, a_s, w_s + wrow * nb, nullptr, r.rows, min((uint32_t)BN, N - n0), 0,
                  r.row0, n0, r.row0 + r.rows};
    if constexpr (GATHER) {
        t.index = g.index + r.row0;
        t.buf_rows = g.src_rows;
    } else {
        t.a += (uint64_t)r.row0 * K;
        t.a_s += (uint64_t)r.row0 * nb;
        t.buf_rows = r.rows;
    }
    gemm_tile<BM, BN, WM, WN, 1, RING, false, GATHER>(t, out, N, K, nb, 0, nullptr, 0, 0, 0);
}

template <int BM, int BN, int WM, int WN, int WG_PER_CU, int RING>
hipError_t launch_grouped(const int8_t *a, const int8_t *w, const float *a_s, const float *w_s, uint16_t *out,
                          const GroupedRows &g, uint32_t n, uint32_t k, hipStream_t s) {
    const uint32_t tiles_n = (uint32_t)div_up(n, BN);
    const uint64_t grid = grouped_row_tiles(g.rows, g.experts, BM) * tiles_n;
    auto kernel = g.index != nullptr ? grouped_kernel<BM, BN, WM, WN, WG_PER_CU, RING, true>
                                     : grouped_kernel<BM, BN, WM, WN, WG_PER_CU, RING, false>;
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(Geo<BM, BN, WM, WN>::kThreads), 0, s, a, w, a_s, w_s, out, g,
                       n, k, tiles_n);
    return hipGetLastError();
}

}  // namespace gemm_kernels

hipError_t launch_grouped_gemm(const int8_t *a, const int8_t *w, const float *a_s, const float *w_s, uint16_t *out,
                               const GroupedRows &g, uint32_t n, uint32_t k, hipStream_t s) {
    using namespace gemm_kernels;
    const uint32_t used = g.rows < g.experts ? g.rows : g.experts;
    const uint32_t mean = g.rows / used;
    if (mean >= 192) return launch_grouped<kGemmTallBM, kGemmBN, 64, 64, 1, 2>(a, w, a_s, w_s, out, g, n, k, s);
    if (mean >= 64) return launch_grouped<kGemmBM, kGemmBN, 64, 64, 2, 2>(a, w, a_s, w_s, out, g, n, k, s);
    return launch_grouped<kGemmSmallTile, kGemmSmallTile, 32, 32, 2, 4>(a, w, a_s, w_s, out, g, n, k, s);
}

}  // namespace bsr
