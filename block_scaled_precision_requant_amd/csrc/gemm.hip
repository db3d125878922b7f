// gemm.hip -- int8 x int8 block-scaled GEMM for gfx950 (m > 16).
//
// Computes out[i,j] = bf16_rne( sum_b fl32(a_s[i,b] * w_s[j,b]) * P[i,j,b] ) with
// P the exact int32 dot product of 32-wide K block b -- the second launch of
// `int8_gemm_faith2_prefill` on page "metrale_model_layers/layers/ops/
// gemm_dense_int8.rs".
//
// The tile itself -- operand staging, matrix-core work, rescale -- is in
// gemm_tile.h; here are the mapping of workgroups to tiles, the K split across
// workgroups and the choice of tile shapes.
#include "gemm_tile.h"

namespace bsr {
namespace gemm_kernels {

template <int BM, int BN, int WM, int WN, int WG_PER_CU, int KG, int RING, bool SPLIT>
__global__ __launch_bounds__(BM * BN / (WM * WN) * 64 * KG, WG_PER_CU) void gemm_kernel(
    const int8_t *__restrict__ a, const int8_t *__restrict__ w, const float *__restrict__ a_s,
    const float *__restrict__ w_s, uint16_t *__restrict__ out, uint32_t M, uint32_t N, uint32_t K,
    uint32_t a_ld, uint32_t a_shift, uint32_t tiles_m, uint32_t tiles_n, float *__restrict__ partial,
    uint64_t pitch, uint32_t slice_stages) {
    uint32_t tm, tn, tile = blockIdx.x, slice = 0;
    if constexpr (SPLIT) {
        slice = blockIdx.x / (tiles_m * tiles_n);
        tile = blockIdx.x % (tiles_m * tiles_n);
    }
    tile_of<BM == kGemmTallBM ? kGemmTallGroupM : kGemmGroupM>(tile, tiles_m, tiles_n, tm, tn);
    const uint32_t m0 = tm * BM, n0 = tn * BN;
    const uint32_t rows_a = min((uint32_t)BM, M - m0);
    const TileArgs t = {a + (uint64_t)m0 * K, w + (uint64_t)n0 * K, a_s + (uint64_t)m0 * a_ld,
                        w_s + (uint64_t)n0 * (K / 32), nullptr, rows_a, min((uint32_t)BN, N - n0), rows_a, m0, n0, M};
    __shared__ __attribute__((aligned(1024))) char lds[TileTraits<BM, BN, WM, WN, KG, RING, SPLIT>::kLds];
    gemm_tile<BM, BN, WM, WN, KG, RING, SPLIT, false>(lds, t, out, N, K, a_ld, a_shift, partial, pitch, slice, slice_stages);
}

// The K slices of a split GEMM: out = bf16_rne(((p_0 + p_1) + p_2) + ...), the
// FP32 slice tiles added in slice order (4 consecutive outputs per lane; each
// slice holds `pitch` floats, m * n rounded up to a multiple of 4).
__global__ __launch_bounds__(256) void split_reduce_kernel(const float *__restrict__ partial,
                                                           uint16_t *__restrict__ out, uint64_t mn, uint64_t pitch,
                                                           uint32_t slices) {
    const uint64_t i = ((uint64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (i >= mn) return;
    typedef float v4f __attribute__((ext_vector_type(4)));
    v4f acc = *reinterpret_cast<const v4f *>(partial + i);
    for (uint32_t sl = 1; sl < slices; ++sl) {
        const v4f v = *reinterpret_cast<const v4f *>(partial + sl * pitch + i);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
    }
    const float r[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (i + j < mn) out[i + j] = f32_to_bf16_rne(r[j]);
}


// Explicit instantiations of every launched shape: clang otherwise left the
// host launch symbols of some instantiations undefined.
#define BSR_GEMM_INST(BM, BN, WM, WN, WGC, KG, RING, SPLIT)                                                 \
    template __global__ void gemm_kernel<BM, BN, WM, WN, WGC, KG, RING, SPLIT>(                             \
        const int8_t *__restrict__, const int8_t *__restrict__, const float *__restrict__,                  \
        const float *__restrict__, uint16_t *__restrict__, uint32_t, uint32_t, uint32_t, uint32_t, uint32_t, \
        uint32_t, uint32_t, float *__restrict__, uint64_t, uint32_t);
BSR_GEMM_INST(256, 128, 64, 64, 1, 1, 2, false)
BSR_GEMM_INST(128, 128, 64, 64, 2, 1, 2, false)
BSR_GEMM_INST(32, 32, 32, 32, 1, 8, 2, false)
BSR_GEMM_INST(32, 32, 32, 32, 2, 4, 2, false)
BSR_GEMM_INST(64, 64, 32, 32, 1, 2, 3, false)
BSR_GEMM_INST(64, 64, 32, 32, 2, 1, 4, false)
BSR_GEMM_INST(64, 64, 32, 32, 2, 1, 4, true)
#undef BSR_GEMM_INST

}  // namespace gemm_kernels

namespace {

using gemm_kernels::gemm_kernel;
using gemm_kernels::split_reduce_kernel;

template <int BM, int BN, int WM, int WN, int WG_PER_CU, int KG = 1, int RING = 2>
hipError_t launch_tiles(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                        const float *w_scale, uint16_t *out, uint32_t m, uint32_t n, uint32_t k,
                        uint32_t a_ld, uint32_t a_shift, hipStream_t s) {
    const uint32_t tiles_m = (uint32_t)div_up(m, BM);
    const uint32_t tiles_n = (uint32_t)div_up(n, BN);
    hipLaunchKernelGGL((gemm_kernel<BM, BN, WM, WN, WG_PER_CU, KG, RING, false>), dim3(tiles_m * tiles_n),
                       dim3(Geo<BM, BN, WM, WN>::kThreads * KG), 0, s, a_i8, w_i8, a_scale, w_scale, out, m, n, k,
                       a_ld, a_shift, tiles_m, tiles_n, nullptr, 0, 0);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale, uint32_t a_ld,
                       uint32_t a_shift, const float *w_scale, uint16_t *out, uint32_t m, uint32_t n,
                       uint32_t k, bool split_k, hipStream_t s) {
    // Grids of at least two 128x128 tiles per CU: one 8-wave 256x128
    // workgroup per CU (LDS 120 KB, 8 waves of about 214 VGPRs) where its
    // 256-row tiling pads M no more than 128-row tiles and K < 2^24, else two
    // 4-wave 128x128 workgroups per CU (LDS 2 x 80 KB, 216 VGPRs), whose
    // barriers fall at different times.  Smaller grids -- every m <= 128,
    // and e.g. m = 512 at n = 4096 -- take 64x64 tiles of four 32x32 waves:
    // four times the workgroups, 1.1-2.5x faster from m = 17 to 1024 on the
    // decode and attention widths; their 4-deep ring (three stages in flight)
    // and 8-block scale stages fit 76 KB of LDS, two workgroups per CU.  Per
    // output the blocks are accumulated in the same order in both, so the bits
    // do not depend on the shape chosen.
    if (gemm_tall_tiles(m, n, k))
        return launch_tiles<kGemmTallBM, kGemmBN, 64, 64, 1>(a_i8, w_i8, a_scale, w_scale, out, m, n, k, a_ld,
                                                             a_shift, s);
    if (gemm_big_tiles(m, n))
        return launch_tiles<kGemmBM, kGemmBN, 64, 64, 2>(a_i8, w_i8, a_scale, w_scale, out, m, n, k, a_ld,
                                                         a_shift, s);
    // Small grids, when K may be split inside a workgroup (its K groups each
    // walk a contiguous range of stages; the FP32 tiles are summed in group
    // order at the end) and K has a stage for every group:
    //  * at most one 32x32 tile per CU: 8 one-wave groups per workgroup
    //    (144 KB of LDS), e.g. m <= 64 at n = 4096, 2x faster than 64x64 tiles;
    //  * at most two: 4 groups, two workgroups per CU (72 KB each) -- also
    //    pads m = 17-32 to 32 rows instead of 64;
    //  * at most one 64x64 tile per CU: 2 groups of four 32x32 waves, each
    //    with a 3-deep ring (two stages in flight while one is computed).
    const uint64_t t32 = div_up(m, kGemmTinyTile) * div_up(n, kGemmTinyTile);
    const uint64_t small_tiles = div_up(m, kGemmSmallTile) * div_up(n, kGemmSmallTile);
    const uint32_t stages = (k / 32 + kGemmStageBlocks - 1) / kGemmStageBlocks;
    if (split_k && t32 <= (uint64_t)kGemmCus && stages >= 8)
        return launch_tiles<kGemmTinyTile, kGemmTinyTile, 32, 32, 1, 8>(a_i8, w_i8, a_scale, w_scale, out, m, n, k,
                                                                         a_ld, a_shift, s);
    if (split_k && t32 <= 2 * (uint64_t)kGemmCus && stages >= 4)
        return launch_tiles<kGemmTinyTile, kGemmTinyTile, 32, 32, 2, 4>(a_i8, w_i8, a_scale, w_scale, out, m, n, k,
                                                                         a_ld, a_shift, s);
    if (split_k && small_tiles <= (uint64_t)kGemmCus && stages >= 2)
        return launch_tiles<kGemmSmallTile, kGemmSmallTile, 32, 32, 1, 2, 3>(a_i8, w_i8, a_scale, w_scale, out, m,
                                                                             n, k, a_ld, a_shift, s);
    return launch_tiles<kGemmSmallTile, kGemmSmallTile, 32, 32, 2, 1, 4>(a_i8, w_i8, a_scale, w_scale, out, m, n,
                                                                         k, a_ld, a_shift, s);
}

hipError_t launch_gemm_split(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                             const float *w_scale, uint16_t *out, uint32_t m, uint32_t n, uint32_t k,
                             float *partial, const SplitPlan &plan, hipStream_t s) {
    // 64 x 64 tiles of four 32 x 32 waves, two workgroups per CU, each with a
    // 4-deep ring (three stages in flight: a slice streams its A and W rows
    // from HBM with ~54 KB per workgroup outstanding)
    const uint32_t tiles_m = (uint32_t)div_up(m, kSplitTile), tiles_n = (uint32_t)div_up(n, kSplitTile);
    const uint32_t grid = tiles_m * tiles_n * plan.slices;
    hipLaunchKernelGGL((gemm_kernel<kSplitTile, kSplitTile, 32, 32, 2, 1, 4, true>), dim3(grid),
                       dim3(Geo<kSplitTile, kSplitTile, 32, 32>::kThreads), 0, s, a_i8, w_i8, a_scale, w_scale,
                       out, m, n, k, k / 32, 0u, tiles_m, tiles_n, partial, plan.pitch, plan.stages);
    if (hipError_t e = hipGetLastError()) return e;
    const uint64_t mn = (uint64_t)m * n;
    hipLaunchKernelGGL(split_reduce_kernel, dim3((uint32_t)div_up(mn, 4 * 256)), dim3(256), 0, s, partial, out, mn,
                       plan.pitch, plan.slices);
    return hipGetLastError();
}

}  // namespace bsr
