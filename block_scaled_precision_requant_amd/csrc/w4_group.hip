// w4_group.hip -- decode GEMV with integer 4-bit weights and a scale and zero
// point per group of k, dense and by expert.
//
// y[i,j] = sum_g s[j,g] * sum_{k in g} x[i,k] * (c[j,k] - z[j,g]).  BF16 with
// the bits 0x4180 | c << 3 is the exact value 16 + c, so a dword of eight codes
// becomes four pairs (elements i and i + 4) with a shift, an AND and an OR
// each.  Per 32 elements two v_mfma_f32_16x16x32_bf16: P = sum x * (16 + c) and
// X = sum x (an all-ones operand, so every column of its tile holds the row
// sums); a group ends with acc += s * (P - (16 + z) * X), everything in FP32.
// The 16 rows of a tile are activation rows, its 16 columns weight rows.
//
// Bound by reading the weight once.  A workgroup owns 16 columns and its waves
// split K, so the weight rows stream straight into registers: a lane loads 16
// bytes (32 codes) of row l % 16, quarter l / 16 of a 128-element chunk, and
// four lane swaps turn the chunk's 4 x 4 dwords so that each MFMA covers 32
// consecutive elements -- one group at least.  A pass of 2 or 4 chunks is in flight while the one
// before it is computed.  Each wave stages the activations of its own pass in
// LDS (in the pairs' order, once per element), so the waves meet only at the
// end, where their sums are added in wave order.
#include "moe_internal.h"

namespace bsr {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Eight codes -> BF16 16 + c, pairs (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w) {
    constexpr uint32_t m = 0x00780078u, base = 0x41804180u;
    const v4i v = {(int)((w << 3 & m) | base), (int)((w >> 1 & m) | base), (int)((w >> 5 & m) | base),
                   (int)((w >> 9 & m) | base)};
    return __builtin_bit_cast(bf16x8, v);
}

// Eight BF16 of an activation row in the same pair order.
__device__ __forceinline__ v4i pair_order(v4i x) {
    return v4i{(int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x07060302u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x07060302u)};
}

// Lane (c, q) holds dword j of quarter q in component j -> dword q of quarter j:
// a 4 x 4 transposition over the four rows of 16 lanes.
__device__ __forceinline__ v4i swap_quarters(v4i w) {
    const auto a = __builtin_amdgcn_permlane16_swap((uint32_t)w.x, (uint32_t)w.y, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap((uint32_t)w.z, (uint32_t)w.w, false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    return v4i{(int)c[0], (int)d[0], (int)c[1], (int)d[1]};
}

// N consecutive elements of BYTES each, as one load wherever they start.
template <int BYTES, int N>
struct Run {
    uint32_t raw[(BYTES * N + 3) / 4];

    __device__ __forceinline__ void load(const void *p, uint64_t at) {
        __builtin_memcpy(raw, static_cast<const uint8_t *>(p) + at * BYTES, BYTES * N);
    }
    // entries from `live` on repeat the last one
    __device__ __forceinline__ void load_some(const void *p, uint64_t at, uint32_t live) {
        const uint8_t *from = static_cast<const uint8_t *>(p) + at * BYTES;
#pragma unroll
        for (int i = 0; i < (BYTES * N + 3) / 4; ++i) raw[i] = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint8_t *e = from + (uint64_t)min((uint32_t)i, live - 1) * BYTES;
            uint32_t v = e[0];
            if constexpr (BYTES == 2) v = *reinterpret_cast<const uint16_t *>(e);
            if constexpr (BYTES == 4) v = *reinterpret_cast<const uint32_t *>(e);
            raw[BYTES * i / 4] |= v << (8 * (BYTES * i % 4));
        }
    }
    __device__ __forceinline__ uint32_t bits(int i) const {
        return raw[BYTES * i / 4] >> (8 * (BYTES * i % 4)) & (BYTES == 4 ? ~0u : (1u << (8 * BYTES % 32)) - 1);
    }
};

template <int STYPE>
__device__ __forceinline__ float scale_value(uint32_t bits) {
    if constexpr (STYPE == 0) return __uint_as_float(bits << 16);
    if constexpr (STYPE == 1) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
    return __uint_as_float(bits);
}

// What a wave holds of one pass.  GPC: groups per 128-element chunk (4, 2, 1),
// or 0 for one scale per weight row.  CT: column tiles.  PC: chunks.
template <int GPC, int STYPE, int CT, int PC>
struct Pass {
    static constexpr int kGroups = GPC > 0 ? GPC * PC : 1;
    v4i w[CT][PC];
    Run<STYPE == 2 ? 4 : 2, kGroups> s[CT];
    Run<1, kGroups> z[CT];
};

struct W4Args {
    const uint16_t *x;
    const uint8_t *w;
    const void *scale;
    const uint8_t *zero;
    uint16_t *out;
    uint32_t n, k, cols, chunks_per_wave;
};

// The wave's chunks of K for one tile of t.rows <= ROWS rows: acc[ct] in MFMA
// layout (lane: column l % 16, rows 4 * (l / 16) + r).  `xs`: this wave's LDS.
template <int GPC, int STYPE, int CT, bool SILU, int ROWS>
__device__ __forceinline__ void w4_rows(const W4Args &p, const GroupedRows &g, const RowTile &t, uint32_t col0,
                                        uint8_t *xs, int lane, int wave, v4f (&acc)[CT]) {
    constexpr int PC = w4g_pass(ROWS <= (int)kW4gFew, CT);
    constexpr uint32_t kPitch = w4g_pitch(PC);
    constexpr int kLoads = ROWS * PC / 4;           // 16-byte activation loads per lane and pass
    constexpr int kRowLoads = PC * kW4gChunk / 8;   // of which a row takes
    const uint32_t c = lane & 15, q = lane >> 4;
    const uint32_t groups = GPC > 0 ? p.k / (kW4gChunk / GPC) : 1;
    const uint32_t chunks = (p.k + kW4gChunk - 1) / kW4gChunk;
    const uint32_t first = wave * p.chunks_per_wave, end = min(chunks, first + p.chunks_per_wave);
    uint64_t wrow[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
        wrow[ct] = (uint64_t)t.expert * p.n + (SILU ? ct * p.cols + min(col0 + c, p.cols - 1)
                                                    : min(col0 + ct * kW4gCols + c, p.cols - 1));

    // activation loads: load i brings 16 bytes of row (64 * i + lane) / kRowLoads
    int32_t xsrc[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint32_t row = (64 * i + lane) / kRowLoads;
        xsrc[i] = row < t.rows ? source_row(g, t.row0 + row) : -1;
    }
    const uint32_t xk = lane % kRowLoads * 8;  // its element within the pass

    using P = Pass<GPC, STYPE, CT, PC>;
    v4i xv[kLoads];
    auto load = [&](P &b, uint32_t chunk) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < PC; ++i) {
            if (chunk + i >= end) break;
            const uint32_t k0 = (chunk + i) * kW4gChunk;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const uint32_t byte = min(k0 / 2 + 16 * q, p.k / 2 - 16);  // past K: any codes, the activations are 0
                b.w[ct][i] = *reinterpret_cast<const v4i *>(p.w + wrow[ct] * (p.k / 2) + byte);
            }
        }
        if constexpr (GPC > 0) {
            const uint32_t g0 = chunk * GPC;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const uint64_t at = wrow[ct] * groups + g0;
                if (g0 + GPC * PC <= groups) {
                    b.s[ct].load(p.scale, at);
                    if (p.zero != nullptr) b.z[ct].load(p.zero, at);
                } else {  // the row's last pass (past K the activations are 0)
                    b.s[ct].load_some(p.scale, at, groups - g0);
                    if (p.zero != nullptr) b.z[ct].load_some(p.zero, at, groups - g0);
                }
            }
        }
    };
    auto load_x = [&](uint32_t chunk) __attribute__((always_inline)) {
        const uint32_t k0 = chunk * kW4gChunk + xk, kend = min(p.k, end * kW4gChunk);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            xv[i] = v4i{0, 0, 0, 0};
            if (xsrc[i] >= 0 && k0 < kend)
                xv[i] = *reinterpret_cast<const v4i *>(p.x + (uint64_t)(uint32_t)xsrc[i] * p.k + k0);
        }
    };
    auto store_x = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t row = (64 * i + lane) / kRowLoads;
            if (row < t.rows) *reinterpret_cast<v4i *>(xs + row * kPitch + xk * 2) = pair_order(xv[i]);
        }
    };

    const v4f none = {0.0f, 0.0f, 0.0f, 0.0f};
    const v4i one4 = {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
    const bf16x8 ones = __builtin_bit_cast(bf16x8, one4);
    v4f psum[CT], xsum = none;  // GPC 0: over the wave's whole range
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) acc[ct] = psum[ct] = none;
    const uint8_t *xa = xs + min(c, t.rows - 1) * kPitch + 16 * q;
    auto compute = [&](const P &b, uint32_t chunk) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < PC; ++i) {
            if (chunk + i >= end) break;
            v4i w[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) w[ct] = swap_quarters(b.w[ct][i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 xv8 = *reinterpret_cast<const bf16x8 *>(xa + i * (kW4gChunk * 2) + j * 64);
                constexpr int per = GPC > 0 ? 4 / GPC : 4;
                if (GPC > 0 && j % per == 0) xsum = none;
                xsum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv8, ones, xsum, 0, 0, 0);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    if (GPC > 0 && j % per == 0) psum[ct] = none;
                    psum[ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv8, codes_to_bf16((uint32_t)w[ct][j]),
                                                                       psum[ct], 0, 0, 0);
                    if (GPC > 0 && j % per == per - 1) {
                        const float s = scale_value<STYPE>(b.s[ct].bits(i * GPC + j / per));
                        const float z = p.zero != nullptr ? (float)b.z[ct].bits(i * GPC + j / per) : 8.0f;
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[ct][r] = fmaf(s, fmaf(-16.0f - z, xsum[r], psum[ct][r]), acc[ct][r]);
                    }
                }
            }
        }
    };

    if (first < end) {
        P b[2];
        load_x(first);
        load(b[0], first);
        for (uint32_t at = first; at < end; at += 2 * PC) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t chunk = at + u * PC;
                if (chunk >= end) break;
                store_x();
                if (chunk + PC < end) {
                    load_x(chunk + PC);
                    load(b[1 - u], chunk + PC);
                }
                compute(b[u], chunk);
            }
        }
    }
    if constexpr (GPC == 0) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const float s = load_f32<STYPE>(p.scale, wrow[ct]);
            const float z = p.zero != nullptr ? (float)p.zero[wrow[ct]] : 8.0f;
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[ct][r] = s * fmaf(-16.0f - z, xsum[r], psum[ct][r]);
        }
    }
}

template <int GPC, int STYPE, int CT, bool SILU>
__global__ __launch_bounds__(kW4gMaxWaves * 64) void w4_group_kernel(W4Args p, GroupedRows g, uint32_t col_tiles,
                                                                     uint32_t wave_bytes) {
    static_assert(!SILU || CT == 2, "a gate and an up tile");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nwaves = blockDim.x >> 6;
    RowTile t = RowTiles(g, kW4gRows, lane).find(blockIdx.x / col_tiles);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.rows == 0) return;
    constexpr uint32_t kOut = SILU ? 1 : CT;  // output column tiles
    const uint32_t col0 = blockIdx.x % col_tiles * (kOut * kW4gCols);
    v4f acc[CT];
    uint8_t *xs = smem + wave * wave_bytes;
    if (t.rows <= kW4gFew)
        w4_rows<GPC, STYPE, CT, SILU, kW4gFew>(p, g, t, col0, xs, lane, wave, acc);
    else
        w4_rows<GPC, STYPE, CT, SILU, kW4gRows>(p, g, t, col0, xs, lane, wave, acc);

    // the waves' sums, added in wave order
    __syncthreads();
    v4f *sums = reinterpret_cast<v4f *>(smem);
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) sums[(wave * CT + ct) * 64 + lane] = acc[ct];
    __syncthreads();
    if (wave != 0) return;
    for (int v = 1; v < nwaves; ++v)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) acc[ct] += sums[(v * CT + ct) * 64 + lane];
#pragma unroll
    for (int ot = 0; ot < (int)kOut; ++ot) {
        const uint32_t col = col0 + ot * kW4gCols + (lane & 15), row = 4 * (lane >> 4);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float y = acc[ot][r];
            if constexpr (SILU) y = y / (1.0f + expf(-y)) * acc[1][r];
            if (row + r < t.rows && col < p.cols)
                p.out[(uint64_t)(t.row0 + row + r) * p.cols + col] = f32_to_bf16_rne(y);
        }
    }
}

template <int STYPE, int CT, bool SILU>
hipError_t launch(const W4Args &p, const GroupedRows &g, uint32_t group, const W4gPlan &plan, hipStream_t s) {
    auto kernel = group == 32    ? w4_group_kernel<4, STYPE, CT, SILU>
                  : group == 64  ? w4_group_kernel<2, STYPE, CT, SILU>
                  : group == 128 ? w4_group_kernel<1, STYPE, CT, SILU>
                                 : w4_group_kernel<0, STYPE, CT, SILU>;
    hipLaunchKernelGGL(kernel, dim3(plan.col_tiles * plan.row_tiles), dim3(64 * plan.waves), plan.lds, s, p, g,
                       plan.col_tiles, plan.wave_bytes);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_group(const uint16_t *x, const uint8_t *w, const void *scale, int scale_type,
                           const uint8_t *zero, uint32_t group, uint16_t *out, const GroupedRows &g, bool silu,
                           uint32_t n, uint32_t k, hipStream_t s) {
    const uint32_t cols = silu ? n / 2 : n;
    const W4gPlan plan = w4_group_plan(g.rows, g.experts, cols, k, silu);
    if (plan.lds > kLdsBytes) return hipErrorInvalidValue;
    const W4Args p = {x, w, scale, zero, out, n, k, cols, plan.chunks_per_wave};
#define BSR_W4G(T)                                                 \
    silu           ? launch<T, 2, true>(p, g, group, plan, s)      \
    : plan.ct == 2 ? launch<T, 2, false>(p, g, group, plan, s)     \
                   : launch<T, 1, false>(p, g, group, plan, s)
    if (scale_type == 0) return BSR_W4G(0);
    if (scale_type == 1) return BSR_W4G(1);
    return BSR_W4G(2);
#undef BSR_W4G
}

}  // namespace bsr
