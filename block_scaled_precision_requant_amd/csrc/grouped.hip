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

// Row tiles of kGemmBM rows in falling order of work, so that the last round of
// workgroups is made of the small ones (6 % less time than in the experts' order on 6016
// rows over 32 uneven experts, n 4096, k 2048, although an expert's remainder then reads its
// weight a second time): first those of more than 64 rows in the experts' order (class 0),
// then an expert's last 33..64 rows (1), then last 1..32 (2).
struct ClassedTiles {
    GroupedRows g;
    int lane;
    uint32_t lo, hi;       // rows of this lane's expert
    uint32_t full, full_incl, last_incl;  // its tiles of class 0, and the inclusive prefixes over the lanes: of
                                          // class 0, and of 1 (low half) and 2 (at most one each per expert)
    uint32_t n0, n1, n2;   // tiles of each class

    __device__ __forceinline__ ClassedTiles(const GroupedRows &g_, int lane_) : g(g_), lane(lane_), n0(0), n1(0), n2(0) {
        for (uint32_t e0 = 0; e0 < g.experts; e0 += 64) {
            load(e0);
            const uint32_t both = __builtin_amdgcn_readlane(last_incl, 63);
            n0 += __builtin_amdgcn_readlane(full_incl, 63);
            n1 += both & 0xFFFFu;
            n2 += both >> 16;
        }
        if (g.experts > 64) load(0);
    }
    __device__ __forceinline__ void load(uint32_t e0) {
        g.range(e0 + lane, lo, hi);
        const uint32_t last = (hi - lo) % kGemmBM;
        full = (hi - lo) / kGemmBM + (last > 64);
        full_incl = full;
        last_incl = (last > 32 && last <= 64 ? 1u : 0u) | (last > 0 && last <= 32 ? 1u << 16 : 0u);
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t x = __shfl_up(full_incl, d), y = __shfl_up(last_incl, d);
            if (lane >= d) {
                full_incl += x;
                last_incl += y;
            }
        }
    }
    __device__ __forceinline__ RowTile find(uint32_t v) {
        const bool whole = v < n0;
        const uint32_t shift = v < n0 + n1 ? 0 : 16;
        v -= whole ? 0 : (shift == 0 ? n0 : n0 + n1);
        for (uint32_t e0 = 0;;) {
            const uint32_t part = (last_incl >> shift) & 0xFFFFu;
            const uint32_t incl = whole ? full_incl : part;
            const uint64_t past = __ballot(incl > v);
            if (past != 0) {
                const int o = __builtin_ctzll(past);
                const uint32_t olo = __builtin_amdgcn_readlane(lo, o), ohi = __builtin_amdgcn_readlane(hi, o);
                const uint32_t first = __builtin_amdgcn_readlane(incl - full, o);
                const uint32_t row0 = whole ? olo + (v - first) * kGemmBM : ohi - (ohi - olo) % kGemmBM;
                return {e0 + o, row0, min((uint32_t)kGemmBM, ohi - row0)};
            }
            v -= __builtin_amdgcn_readlane(incl, 63);
            e0 += 64;
            if (e0 >= g.experts) return {0, 0, 0};
            load(e0);
        }
    }
};

// Workgroup -> (row tile, column tile).  Tiles are walked in groups of
// kGemmGroupM row tiles, down the rows first; each XCD takes runs of kRun
// consecutive tiles in turn, so that a run shares A and W rows in the XCD's L2
// while the work of every part of the list is spread over all XCDs (one run
// per XCD, as the dense GEMM has it, gives some XCDs the full tiles and others
// the experts' remainders: 7 % slower on the 6016 rows above; runs of 64, 128
// and 256 tiles level to 5 % slower).
constexpr uint32_t kRun = 32;
__device__ __forceinline__ void grouped_tile_of(uint32_t wg, uint32_t tiles_m, uint32_t tiles_n, uint32_t &tm,
                                                uint32_t &tn) {
    const uint32_t total = tiles_m * tiles_n, whole = total / (kXcds * kRun);
    const uint32_t x = wg % kXcds, j = wg / kXcds;
    uint32_t v;
    if (j / kRun < whole) {
        v = (j / kRun * kXcds + x) * kRun + j % kRun;
    } else {
        const uint32_t left = total - whole * kXcds * kRun, q = left / kXcds, r = left % kXcds;
        v = whole * kXcds * kRun + x * q + min(x, r) + (j - whole * kRun);
    }
    const uint32_t per_group = kGemmGroupM * tiles_n;
    const uint32_t first_m = v / per_group * kGemmGroupM;
    const uint32_t gsize = min(tiles_m - first_m, (uint32_t)kGemmGroupM);
    tm = first_m + v % per_group % gsize;
    tn = v % per_group / gsize;
}

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
    ClassedTiles rt(g, threadIdx.x & 63);
    // (overlapping ranges could ask for more tiles than the grid has: those are not computed)
    const uint32_t tiles_m = min(rt.n0 + rt.n1 + rt.n2, gridDim.x / tiles_n);
    if (blockIdx.x >= tiles_m * tiles_n) return;
    uint32_t tm, tn;
    grouped_tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
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
