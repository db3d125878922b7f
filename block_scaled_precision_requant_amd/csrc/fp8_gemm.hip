// fp8_gemm.hip -- the FP8 products with many rows, dense and grouped by expert.
//
// out[i,j] = sum_b fl32(a_s[i,b] * w_s[j/128,b]) * P[i,j,b], P the dot product of
// block b.  One v_mfma_f32_16x16x128_f8f6f4 covers a whole scale block of 16 x 16
// outputs; the weight is its row operand, so a lane holds four columns of one
// activation row and a block ends with one FMA per output by a scale that is one
// product per lane and 16 rows.
//
// A stage is one block: 128 bytes of every A and W row of the tile, copied straight
// from global memory into LDS, the next stage in flight while one is computed.  The
// activations' scales come four blocks (16 bytes of a row) at a time.
#include "fp8_internal.h"
#include "gemm_tile.h"

namespace bsr {
namespace fp8_kernels {

template <int BM, int BN, int WM, int WN>
struct Fp8Geo {
    static constexpr int kTM = WM / 16, kTN = WN / 16;  // 16 x 16 MFMA tiles per wave
    static constexpr int kWavesN = BN / WN, kWaves = BM / WM * kWavesN;
    static constexpr int kSegA = BM / 8 / kWaves, kSegW = BN / 8 / kWaves;  // 1 KB copies per wave and stage
    static constexpr int kSegS = (BM / 16 + kWaves - 1) / kWaves;           // 256-byte scale copies per four stages
    static_assert(BM / 8 % kWaves == 0 && BN / 8 % kWaves == 0, "whole copies");
    static constexpr uint32_t kStage = (BM + BN) * kFp8Block;
    static constexpr uint32_t kScales = BM * 4 * 4;
    static constexpr uint32_t kLds = 2 * (kStage + kScales);
};

// One tile.  rows_a, cols: valid rows and output columns; row0: first output row.
struct Fp8Tile {
    const uint8_t *a, *w, *w_up;  // first row of each (a: with GATHER the whole operand)
    const float *a_s, *w_s, *w_s_up;  // w_s: row of blocks of the first weight row
    const int32_t *index;
    uint32_t rows_a, buf_rows, cols, row0, col0;
};

template <int BM, int BN, int WM, int WN, bool SILU, bool GATHER>
__device__ __forceinline__ void fp8_tile(char *lds, const Fp8Tile &t, uint16_t *__restrict__ out, uint32_t out_ld,
                                         uint32_t k, bool wide) {
    using G = Fp8Geo<BM, BN, WM, WN>;
    constexpr int TM = G::kTM, TN = G::kTN;
    constexpr uint32_t kWaveCols = SILU ? WN / 2 : WN;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / G::kWavesN, wn = wave % G::kWavesN;
    const uint32_t c = lane & 15, q = lane >> 4, nb = k / kFp8Block;

    const auto ra = __builtin_amdgcn_make_buffer_rsrc((void *)t.a, (short)0, (int)(t.buf_rows * k), kRsrcWord3);
    const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)t.a_s, (short)0, (int)(t.buf_rows * nb * 4), kRsrcWord3);
    const auto rw = __builtin_amdgcn_make_buffer_rsrc((void *)t.w, (short)0, (int)(t.cols * k), kRsrcWord3);
    const auto ru = __builtin_amdgcn_make_buffer_rsrc((void *)t.w_up, (short)0, (int)(t.cols * k), kRsrcWord3);
    uint32_t oa[G::kSegA], ow[G::kSegW], os[G::kSegS];
    auto source = [&](uint32_t row) -> uint32_t {  // offset, in rows, of tile row `row`; ~0: zeros
        if (row >= t.rows_a) return ~0u;
        if constexpr (!GATHER) return row;
        const uint32_t i = (uint32_t)t.index[row];
        return i < t.buf_rows ? i : ~0u;
    };
#pragma unroll
    for (int i = 0; i < G::kSegA; ++i) {
        const uint32_t row = (wave + i * G::kWaves) * 8 + lane / 8, src = source(row);
        oa[i] = src == ~0u ? kPastEnd : src * k + (((lane & 7) ^ chunk_swz(row)) << 4);
    }
#pragma unroll
    for (int i = 0; i < G::kSegW; ++i) {
        const uint32_t row = (wave + i * G::kWaves) * 8 + lane / 8;
        // with the SiLU product a wave's columns are WN / 2 gates, then their ups
        const uint32_t col = SILU ? row / WN * kWaveCols + row % kWaveCols : row;
        ow[i] = col * k + (((lane & 7) ^ chunk_swz(row)) << 4);
    }
#pragma unroll
    for (int i = 0; i < G::kSegS; ++i) {
        const uint32_t row = (wave + i * G::kWaves) * 16 + lane / 4, src = row < BM ? source(row) : ~0u;
        os[i] = src == ~0u ? kPastEnd : src * nb * 4 + (lane & 3) * 4;
    }
    auto copy_stage = [&](uint32_t b) __attribute__((always_inline)) {
        char *to = lds + (b & 1) * G::kStage;
#pragma unroll
        for (int i = 0; i < G::kSegA; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void *)(to + (wave + i * G::kWaves) * 1024), 16, oa[i],
                                                     b * kFp8Block, 0, 0);
#pragma unroll
        for (int i = 0; i < G::kSegW; ++i) {
            const uint32_t row = (wave + i * G::kWaves) * 8;
            const bool up = SILU && row % WN >= kWaveCols;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                up ? ru : rw, (lds_void *)(to + BM * kFp8Block + (wave + i * G::kWaves) * 1024), 16, ow[i], b * kFp8Block, 0,
                0);
        }
    };
    // scales of the blocks from b on (b a multiple of 4; those past K are other
    // numbers or 0, and not used)
    auto copy_scales = [&](uint32_t b) __attribute__((always_inline)) {
        char *to = lds + 2 * G::kStage + (b >> 2 & 1) * G::kScales;
#pragma unroll
        for (int i = 0; i < G::kSegS; ++i) {
            const int seg = wave + i * G::kWaves;
            if (BM / 16 % G::kWaves == 0 || seg < BM / 16)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_void *)(to + seg * 256), 4, os[i], b * 4, 0, 0);
        }
    };

    // operand offsets: lane l reads row l % 16 of its tile, 16-byte chunks 2 (l / 16) and the next
    const uint32_t sw = chunk_swz(c);
    const uint32_t c0 = ((2 * q) ^ sw) << 4, c1 = ((2 * q + 1) ^ sw) << 4;
    const uint32_t row_a = (wm * WM + c) * kFp8Block, row_w = BM * kFp8Block + (wn * WN + c) * kFp8Block;
    auto operand = [&](const char *row) __attribute__((always_inline)) -> v8i {
        return __builtin_shufflevector(*reinterpret_cast<const v4i *>(row + c0), *reinterpret_cast<const v4i *>(row + c1), 0, 1,
                                       2, 3, 4, 5, 6, 7);
    };
    // the weight's scales of 64 blocks, one per lane
    const uint32_t first_col = t.col0 + wn * kWaveCols;
    const float *ws = t.w_s + (uint64_t)((t.col0 % kFp8Block + wn * kWaveCols) / kFp8Block) * nb;
    const float *wsu = t.w_s_up + (uint64_t)((t.col0 % kFp8Block + wn * kWaveCols) / kFp8Block) * nb;
    const bool any = wn * kWaveCols < t.cols;  // (a wave past the last column has no scale block)
    float wsv = 0.0f, wsuv = 0.0f;

    v4f acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = v4f{0, 0, 0, 0};

    copy_scales(0);
    copy_stage(0);
    for (uint32_t b = 0; b < nb; ++b) {
        if (b % 64 == 0) {
            const uint32_t at = min(b + lane, nb - 1);
            if (any) {
                wsv = ws[at];
                if constexpr (SILU) wsuv = wsu[at];
            }
            asm volatile("" : "+v"(wsv), "+v"(wsuv));  // waited for here, not in every turn of the loop
        }
        wait_copies<0>();
        stage_barrier();
        if (b + 1 < nb) copy_stage(b + 1);
        if (b % 4 == 0 && b + 4 < nb) copy_scales(b + 4);
        const char *st = lds + (b & 1) * G::kStage;
        const float *as = reinterpret_cast<const float *>(lds + 2 * G::kStage + (b >> 2 & 1) * G::kScales) + b % 4;
        const float s_w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv), b % 64));
        const float s_u = SILU ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsuv), b % 64)) : s_w;
        v8i wf[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) wf[j] = operand(st + row_w + j * 16 * kFp8Block);
        v4f p[2][TN];
        v8i af = operand(st + row_a);
#pragma unroll
        for (int j = 0; j < TN; ++j) p[0][j] = fp8_dot16(wf[j], af);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            if (i + 1 < TM) {
                af = operand(st + row_a + (i + 1) * 16 * kFp8Block);
#pragma unroll
                for (int j = 0; j < TN; ++j) p[(i + 1) & 1][j] = fp8_dot16(wf[j], af);
            }
            const float sa = as[(wm * WM + i * 16 + c) * 4];
            const float s = sa * s_w, s2 = SILU ? sa * s_u : s;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[i][j][r] = fmaf(p[i & 1][j][r], SILU && j >= TN / 2 ? s2 : s, acc[i][j][r]);
        }
        // (a stage's reads have returned before its compute ends, which the next barrier stands behind)
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) asm volatile("" : "+v"(acc[i][j]));
    }

#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const uint32_t row = wm * WM + i * 16 + c;
        if (row >= t.rows_a) continue;
#pragma unroll
        for (int j = 0; j < (SILU ? TN / 2 : TN); ++j) {
            v4f v = acc[i][j];
            if constexpr (SILU)
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = silu_product(v[r], acc[i][j + TN / 2][r]);
            store4(out, t.row0 + row, first_col + j * 16 + 4 * q, out_ld, v, wide);
        }
    }
}

// Workgroup -> row tile (of g, none across two experts) and column tile.
template <int BM, int BN, int WM, int WN, bool SILU, bool GATHER>
__global__ __launch_bounds__((Fp8Geo<BM, BN, WM, WN>::kWaves) * 64, 2) void fp8_gemm_kernel(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ w, const float *__restrict__ a_s,
    const float *__restrict__ w_s, uint16_t *__restrict__ out, GroupedRows g, uint32_t n, uint32_t k,
    uint32_t tiles_m, uint32_t tiles_n, bool wide) {
    __shared__ __attribute__((aligned(1024))) char lds[Fp8Geo<BM, BN, WM, WN>::kLds];
    constexpr uint32_t kCols = SILU ? BN / 2 : BN;
    uint32_t tm, tn;
    tile_of<4>(blockIdx.x, tiles_m, tiles_n, tm, tn);
    RowTile r = RowTiles(g, BM, threadIdx.x & 63).find(tm);
    r.expert = __builtin_amdgcn_readfirstlane(r.expert);
    r.row0 = __builtin_amdgcn_readfirstlane(r.row0);
    r.rows = __builtin_amdgcn_readfirstlane(r.rows);
    if (r.rows == 0) return;
    const uint32_t half = n / 2, cols = SILU ? half : n, nb = k / kFp8Block, blocks = (n + kFp8Block - 1) / kFp8Block;
    const uint32_t col0 = __builtin_amdgcn_readfirstlane(tn * kCols);
    const uint64_t wrow = (uint64_t)r.expert * n + col0, wblock = (uint64_t)r.expert * blocks + col0 / kFp8Block;
    Fp8Tile t = {a, w + wrow * k, w + (wrow + half) * k, a_s, w_s + wblock * nb, w_s + (wblock + half / kFp8Block) * nb,
                 nullptr, r.rows, r.rows, min(kCols, cols - col0), r.row0, col0};
    if constexpr (GATHER) {
        t.index = g.index + r.row0;
        t.buf_rows = __builtin_amdgcn_readfirstlane(g.src_rows);
    } else {
        t.a += (uint64_t)r.row0 * k;
        t.a_s += (uint64_t)r.row0 * nb;
    }
    fp8_tile<BM, BN, WM, WN, SILU, GATHER>(lds, t, out, cols, k, wide);
}

template <int BM, int BN, int WM, int WN>
void launch_tile(const Fp8Args &p, const Fp8Choice &c, hipStream_t s) {
    const uint32_t cols = p.silu ? p.n / 2 : p.n;
    const bool wide = cols % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % 8 == 0;
    auto kernel = p.silu ? (p.rows.index ? fp8_gemm_kernel<BM, BN, WM, WN, true, true> : fp8_gemm_kernel<BM, BN, WM, WN, true, false>)
                         : (p.rows.index ? fp8_gemm_kernel<BM, BN, WM, WN, false, true>
                                         : fp8_gemm_kernel<BM, BN, WM, WN, false, false>);
    hipLaunchKernelGGL(kernel, dim3(c.tiles_m * c.tiles_n), dim3(Fp8Geo<BM, BN, WM, WN>::kWaves * 64), 0, s, p.a, p.w, p.a_s,
                       p.w_s, p.out, p.rows, p.n, p.k, c.tiles_m, c.tiles_n, wide);
}

}  // namespace fp8_kernels

hipError_t launch_fp8_gemm(const Fp8Args &p, hipStream_t s) {
    const Fp8Choice c = fp8_choice(p.rows.rows, p.rows.experts, p.n, p.k, p.silu, p.rows.offsets != nullptr);
    if (c.stream) return launch_fp8_stream(p, c.plan, s);
    if (c.bm == kFp8Tall)
        fp8_kernels::launch_tile<256, 256, 128, 64>(p, c, s);
    else
        fp8_kernels::launch_tile<128, 128, 64, 64>(p, c, s);
    return hipGetLastError();
}

}  // namespace bsr
