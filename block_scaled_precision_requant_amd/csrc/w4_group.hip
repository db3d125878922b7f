// w4_group.hip -- decode GEMV with integer 4-bit weights and a scale and zero
// point per group of k, dense and by expert.
//
// y[i,j] = sum_g s[j,g] * sum_{k in g} x[i,k] * (c[j,k] - z[j,g]).  BF16 with
// the bits 0x4180 | c << 3 is the exact value 16 + c, so a dword of eight codes
// becomes four pairs (elements i and i + 4) with a shift, an AND and an OR
// each.  Per 32 elements two v_mfma_f32_16x16x32_bf16: P = sum x * (16 + c) and
// X = sum x (an all-ones operand, so every column of its tile holds the row
// sums); a group ends with acc += s * (P - (16 + z) * X).  The 16 rows of a
// tile are activation rows, its 16 columns weight rows.
#include "moe_internal.h"

namespace bsr {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kRows = 16, kCols = 64;

// Eight codes -> BF16 16 + c, pairs (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ v4i codes_to_bf16(uint32_t w) {
    constexpr uint32_t m = 0x00780078u, base = 0x41804180u;
    return v4i{(int)((w << 3 & m) | base), (int)((w >> 1 & m) | base), (int)((w >> 5 & m) | base),
               (int)((w >> 9 & m) | base)};
}

// Eight BF16 of an activation row in the same pair order.
__device__ __forceinline__ v4i pair_order(v4i x) {
    return v4i{(int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x07060302u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x07060302u)};
}

template <int STYPE>
__device__ __forceinline__ v4f dot_column(const uint16_t *x, const uint8_t *w, const void *scale, const uint8_t *zero,
                                          uint64_t wrow, int32_t src, uint32_t group, uint32_t k, uint32_t q) {
    const v4i ones = {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
    const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t *wp = w + wrow * (k / 2) + 4 * q;
    const uint16_t *xp = x + (uint64_t)max(src, 0) * k + 8 * q;
    const uint32_t per = group / 32, groups = k / group;
    v4f acc = none;
    for (uint32_t gi = 0; gi < groups; ++gi) {
        v4f p = none, sx = none;
        for (uint32_t b = gi * per; b < (gi + 1) * per; ++b) {
            v4i xv = pair_order(*reinterpret_cast<const v4i *>(xp + 32 * (uint64_t)b));
            if (src < 0) xv = v4i{0, 0, 0, 0};
            const v4i wv = codes_to_bf16(*reinterpret_cast<const uint32_t *>(wp + 16 * (uint64_t)b));
            p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv), __builtin_bit_cast(bf16x8, wv),
                                                        p, 0, 0, 0);
            sx = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, xv),
                                                         __builtin_bit_cast(bf16x8, ones), sx, 0, 0, 0);
        }
        const float s = load_f32<STYPE>(scale, wrow * groups + gi);
        const float z = -(16.0f + (zero != nullptr ? (float)zero[wrow * groups + gi] : 8.0f));
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] = fmaf(s, fmaf(z, sx[r], p[r]), acc[r]);
    }
    return acc;
}

template <int STYPE>
__global__ __launch_bounds__(256) void w4_group_kernel(const uint16_t *__restrict__ x, const uint8_t *__restrict__ w,
                                                       const void *__restrict__ scale,
                                                       const uint8_t *__restrict__ zero, uint32_t group,
                                                       uint16_t *__restrict__ out, GroupedRows g, uint32_t n,
                                                       uint32_t k, uint32_t col_tiles, bool silu) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const RowTile t = RowTiles(g, kRows, lane).find(blockIdx.x / col_tiles);
    if (t.rows == 0) return;
    const uint32_t c = lane & 15, q = lane >> 4;
    const uint32_t cols = silu ? n / 2 : n;
    const uint32_t col = (blockIdx.x % col_tiles) * kCols + wave * 16 + c;
    const int32_t src = c < t.rows ? source_row(g, t.row0 + c) : -1;
    const uint64_t wrow = (uint64_t)t.expert * n + min(col, cols - 1);
    v4f y = dot_column<STYPE>(x, w, scale, zero, wrow, src, group, k, q);
    if (silu) {
        const v4f up = dot_column<STYPE>(x, w, scale, zero, wrow + cols, src, group, k, q);
#pragma unroll
        for (int r = 0; r < 4; ++r) y[r] = y[r] / (1.0f + expf(-y[r])) * up[r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * q + r < t.rows && col < cols) out[(uint64_t)(t.row0 + 4 * q + r) * cols + col] = f32_to_bf16_rne(y[r]);
}

}  // namespace

hipError_t launch_w4_group(const uint16_t *x, const uint8_t *w, const void *scale, int scale_type,
                           const uint8_t *zero, uint32_t group, uint16_t *out, const GroupedRows &g, bool silu,
                           uint32_t n, uint32_t k, hipStream_t s) {
    if (group == 0) group = k;
    const uint32_t col_tiles = (uint32_t)div_up(silu ? n / 2 : n, kCols);
    const uint64_t grid = grouped_row_tiles(g.rows, g.experts, kRows) * col_tiles;
    auto kernel = scale_type == 0 ? w4_group_kernel<0> : (scale_type == 1 ? w4_group_kernel<1> : w4_group_kernel<2>);
    hipLaunchKernelGGL(kernel, dim3((uint32_t)grid), dim3(256), 0, s, x, w, scale, zero, group, out, g, n, k, col_tiles,
                       silu);
    return hipGetLastError();
}

}  // namespace bsr
