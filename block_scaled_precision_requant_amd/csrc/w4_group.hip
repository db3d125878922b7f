// w4_group.hip -- decode GEMV with integer 4-bit weights and a scale and zero
// point per group of k, dense and by expert.
//
// y[i,j] = sum_g s[j,g] * sum_{k in g} x[i,k] * (c[j,k] - z[j,g]).  BF16 with
// the bits 0x4180 | c << 3 is the exact value 16 + c, so a dword of eight codes
// becomes four pairs (elements i and i + 4) with a shift, an AND and an OR
// each.  Per 32 elements two v_mfma_f32_16x16x32_bf16: P = sum x * (16 + c) and
// X = sum x (an all-ones operand, so every column of its tile holds the row
// sums); a group ends with acc += s * (P - (16 + z) * X), everything in FP32.
// One scale per weight row ends every 128 elements the same way: P and X over
// all of K, far above their difference, would round 3 to 6 times as coarsely.
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
//
// MI355X, weights from HBM: one row, N 14336, K 4096, groups of 128 (30.8 MB) 10.5 us; 16
// rows, N 4096, K 14336, groups of 32 (33.6 MB) 17.6 us (13.2 where the weights are in the
// 256 MB cache): there vector issue is half of the waves' time, waiting the other half; a
// CU takes 131 KB of weight and 459 KB of activations through its L1.
#include "moe_internal.h"

namespace bsr {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Sums are held 2^-kDown times as large: 128 elements of any finite BF16 times
// |c - z| <= 255 then stay under binary32's largest value (255 * 128 < 2^15),
// and powers of two change no rounding above its smallest.
constexpr int kDown = 15;

// Eight codes -> BF16 (16 + c) * 2^-kDown, pairs (0,4) (1,5) (2,6) (3,7); mask = 0x00780078.
__device__ __forceinline__ bf16x8 codes_to_bf16(uint32_t w, uint32_t mask) {
    constexpr uint32_t base = 0x41804180u - kDown * 0x00800080u;
    const v4i v = {(int)((w << 3 & mask) | base), (int)((w >> 1 & mask) | base), (int)((w >> 5 & mask) | base),
                   (int)((w >> 9 & mask) | base)};
    return __builtin_bit_cast(bf16x8, v);
}

// Eight BF16 of an activation row in the same pair order.
__device__ __forceinline__ v4i pair_order(v4i x) {
    return v4i{(int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x07060302u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x05040100u),
               (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x07060302u)};
}

// N consecutive elements of BYTES each, loaded as wide as they come wherever
// they start (words and vectors of any alignment; held as words, since an
// array filled byte-wise would live in memory).
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint16_t u16_any __attribute__((aligned(1)));

template <int BYTES, int N>
struct Run {
    static constexpr int kBytes = BYTES * N, kWords = (kBytes + 3) / 4;
    uint32_t raw[kWords];

    __device__ __forceinline__ void load(const uint8_t *from) {
        if constexpr (kBytes == 1) raw[0] = *from;
        if constexpr (kBytes == 2) raw[0] = *reinterpret_cast<const u16_any *>(from);
        if constexpr (kBytes == 4) raw[0] = *reinterpret_cast<const u32_any *>(from);
        if constexpr (kBytes == 8) {
            const u32x2_any v = *reinterpret_cast<const u32x2_any *>(from);
            raw[0] = v.x;
            raw[1] = v.y;
        }
        if constexpr (kBytes >= 16) {
            static_assert(kBytes % 16 == 0, "whole 16-byte words");
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const u32x4_any v = *reinterpret_cast<const u32x4_any *>(from + 4 * i);
                raw[i] = v.x;
                raw[i + 1] = v.y;
                raw[i + 2] = v.z;
                raw[i + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void fill(uint32_t word) {
#pragma unroll
        for (int i = 0; i < kWords; ++i) raw[i] = word;
    }
    // the first `live` entries; the others are 0
    __device__ __forceinline__ void load_some(const uint8_t *from, uint32_t live) {
#pragma unroll
        for (int i = 0; i < (BYTES * N + 3) / 4; ++i) raw[i] = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if ((uint32_t)i >= live) break;
            uint32_t v = from[i * BYTES];
            if constexpr (BYTES == 2) v = *reinterpret_cast<const u16_any *>(from + i * BYTES);
            if constexpr (BYTES == 4) v = *reinterpret_cast<const u32_any *>(from + i * BYTES);
            raw[BYTES * i / 4] |= v << (8 * (BYTES * i % 4));
        }
    }
    __device__ __forceinline__ uint32_t bits(int i) const {
        return raw[BYTES * i / 4] >> (8 * (BYTES * i % 4)) & (BYTES == 4 ? ~0u : (1u << (8 * BYTES % 32)) - 1);
    }
};

template <int STYPE>
constexpr uint32_t kScaleBytes = STYPE == 2 ? 4 : 2;

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
    Run<kScaleBytes<STYPE>, kGroups> s[CT];
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

// The wave's chunks of K for one tile of t.rows <= ROWS rows: 2^-kDown acc[ct] in MFMA
// layout (lane: column l % 16, rows 4 * (l / 16) + r).  `xs`: this wave's LDS.
template <int GPC, int STYPE, int CT, bool SILU, int ROWS>
__device__ __forceinline__ void w4_rows(const W4Args &p, const GroupedRows &g, const RowTile &t, uint32_t col0,
                                        uint8_t *xs, int lane, int wave, v4f (&acc)[CT]) {
    constexpr int PC = w4g_pass(CT, GPC), XC = w4g_stage(ROWS, CT, GPC);  // chunks per pass, and per staging of x
    constexpr uint32_t kPitch = w4g_pitch(XC);
    constexpr int kLoads = ROWS * XC / 4;           // 16-byte activation loads per lane and staging
    constexpr int kRowLoads = XC * kW4gChunk / 8;   // of which a row takes
    static_assert(PC % XC == 0, "whole stagings per pass");
    const uint32_t c = lane & 15, q = lane >> 4;
    const uint32_t groups = GPC > 0 ? p.k / (kW4gChunk / GPC) : 1;
    const uint32_t chunks = (p.k + kW4gChunk - 1) / kW4gChunk;
    const uint32_t first = wave * p.chunks_per_wave, end = min(chunks, first + p.chunks_per_wave);
    // Addresses: a descriptor or base pointer that is the same in all lanes, a
    // 32-bit offset per lane that stays, and the pass's offset as a scalar.
    // Weight rows past the last column read as 0; scalar offsets stay inside a
    // row, so that a buffer's end bounds every load.
    __amdgpu_buffer_rsrc_t rw[CT];
    const uint8_t *sbase[CT], *zbase[CT];
    uint32_t srow[CT];  // scale row within the tile
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        // (CT 2: a second tile past the end reads the last row and is not written)
        const uint32_t c0 = SILU ? col0 : col0 + ct * kW4gCols;
        const uint32_t live = c0 < p.cols ? min(p.cols - c0, kW4gCols) : 1;
        const uint64_t row = (uint64_t)t.expert * p.n + (SILU ? ct * p.cols : 0) + min(c0, p.cols - 1);
        rw[ct] = __builtin_amdgcn_make_buffer_rsrc((void *)(p.w + row * (p.k / 2)), (short)0, (int)(live * (p.k / 2)),
                                                   kRsrcWord3);
        sbase[ct] = static_cast<const uint8_t *>(p.scale) + row * groups * kScaleBytes<STYPE>;
        zbase[ct] = p.zero + row * groups;
        srow[ct] = min(c, live - 1);
    }
    const uint32_t wo = c * (p.k / 2) + 16 * q;

    // activation loads: load i brings 16 bytes of row (64 * i + lane) / kRowLoads
    const __amdgpu_buffer_rsrc_t rx =
        __builtin_amdgcn_make_buffer_rsrc((void *)p.x, (short)0, (int)(g.src_rows * p.k * 2), kRsrcWord3);
    uint32_t xo[kLoads];
    const uint32_t xk = lane % kRowLoads * 8;  // its element within the staging
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint32_t row = (64 * i + lane) / kRowLoads;
        const int32_t src = row < t.rows ? source_row(g, t.row0 + row) : -1;
        xo[i] = src >= 0 ? ((uint32_t)src * p.k + xk) * 2 : kPastEnd;
    }

    // A pass comes in whole (all its chunks in this wave's range and inside K)
    // or, as the wave's last one, in part: then chunks past the range are
    // skipped, and past K the activations are 0 and codes and scales any.
    using P = Pass<GPC, STYPE, CT, PC>;
    v4i xv[kLoads];
    auto load = [&](P &b, uint32_t chunk, bool part) __attribute__((always_inline)) {
        if constexpr (GPC > 0) {
            const uint32_t g0 = chunk * GPC;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const uint8_t *sp = sbase[ct] + g0 * kScaleBytes<STYPE> + srow[ct] * (groups * kScaleBytes<STYPE>);
                const uint8_t *zp = zbase[ct] + g0 + srow[ct] * groups;
                if (!part || g0 + GPC * PC <= groups) {
                    b.s[ct].load(sp);
                    if (p.zero != nullptr) b.z[ct].load(zp);
                } else {
                    b.s[ct].load_some(sp, groups - g0);
                    if (p.zero != nullptr) b.z[ct].load_some(zp, groups - g0);
                }
                if (p.zero == nullptr) b.z[ct].fill(0x08080808u);
            }
        }
#pragma unroll
        for (int i = 0; i < PC; ++i)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                b.w[ct][i] = load16(rw[ct], wo, min(chunk + i, part ? chunks - 1 : ~0u) * (kW4gChunk / 2));
    };
    auto load_x = [&](uint32_t chunk, bool part) __attribute__((always_inline)) {
        const bool live = !part || chunk * kW4gChunk + xk < p.k;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (ROWS <= (int)kW4gFew && 64u * i / kRowLoads >= t.rows) break;
            xv[i] = load16(rx, live ? xo[i] : kPastEnd, chunk * (kW4gChunk * 2));
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
    constexpr int kOnes = 0x3F803F80 - kDown * 0x00800080;  // 2^-kDown, twice
    const bf16x8 ones = __builtin_bit_cast(bf16x8, v4i{kOnes, kOnes, kOnes, kOnes});
    uint32_t mask = 0x00780078u;  // in a register of its own: v_and_or_b32 takes one constant
    asm("" : "+v"(mask));
    v4f psum[CT], xsum;
    float row_scale[CT], row_zero[CT];  // GPC 0
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        acc[ct] = none;
        if constexpr (GPC == 0) {
            row_scale[ct] = load_f32<STYPE>(sbase[ct], srow[ct]);
            row_zero[ct] = p.zero != nullptr ? (float)zbase[ct][srow[ct]] : 8.0f;
        }
    }
    const uint8_t *xa = xs + min(c, t.rows - 1) * kPitch + 16 * q;
    // chunks [i0, i0 + XC) of a pass, whose activations are staged
    auto compute = [&](const P &b, int i0, uint32_t live) __attribute__((always_inline)) {
#pragma unroll
        for (int ii = 0; ii < XC; ++ii) {
            const int i = i0 + ii;
            if ((uint32_t)i >= live) break;
            asm volatile("" ::: "memory");  // a chunk's reads stay with it: bounds live registers
            v4i w[CT];
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) w[ct] = swap_quarters(b.w[ct][i]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bf16x8 xv8 = *reinterpret_cast<const bf16x8 *>(xa + ii * (kW4gChunk * 2) + j * 64);
                constexpr int per = GPC > 0 ? 4 / GPC : 4;
                if (j % per == 0) xsum = none;
                xsum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv8, ones, xsum, 0, 0, 0);
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) {
                    if (j % per == 0) psum[ct] = none;
                    psum[ct] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv8, codes_to_bf16((uint32_t)w[ct][j], mask),
                                                                       psum[ct], 0, 0, 0);
                    if (j % per == per - 1) {
                        float s, z;
                        if constexpr (GPC > 0) {
                            s = scale_value<STYPE>(b.s[ct].bits(i * GPC + j / per));
                            z = (float)b.z[ct].bits(i * GPC + j / per);
                        } else {
                            s = row_scale[ct], z = row_zero[ct];
                        }
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[ct][r] = fmaf(s, fmaf(-16.0f - z, xsum[r], psum[ct][r]), acc[ct][r]);
                    }
                }
            }
        }
    };
    // One whole pass; `more`: the next one is whole too, and its loads go out
    // before this one is computed.  Loads return in order, so a staging's
    // activations are asked for before the next pass's weights wherever they
    // are needed before them.  (more is a constant at each call: a load that
    // may or may not have been issued would make every later wait the longer one.)
    auto pass = [&](P &b, P &next, uint32_t chunk, bool more) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < PC; i += XC) {
            store_x();
            if (i + XC < PC)
                load_x(chunk + i + XC, false);
            else if (more)
                load_x(chunk + PC, false);
            if (i == 0 && more) load(next, chunk + PC, false);
            compute(b, i, PC);
        }
    };
    const uint32_t whole = min(end, p.k / kW4gChunk);           // chunks before this one are whole
    const uint32_t passes = first < whole ? (whole - first) / PC : 0;
    P b0, b1;
    uint32_t chunk = first;
    if (passes > 0) {
        load_x(chunk, false);
        load(b0, chunk, false);
        const uint32_t last = first + (passes - 1) * PC;
        for (;;) {
            if (chunk == last) {
                pass(b0, b1, chunk, false);
                break;
            }
            pass(b0, b1, chunk, true);
            chunk += PC;
            if (chunk == last) {
                pass(b1, b0, chunk, false);
                break;
            }
            pass(b1, b0, chunk, true);
            chunk += PC;
        }
        chunk += PC;
    }
    if (chunk < end) {
        load_x(chunk, true);
        load(b0, chunk, true);
#pragma unroll
        for (int i = 0; i < PC; i += XC) {
            if (chunk + i >= end) break;
            if (i > 0) load_x(chunk + i, true);
            store_x();
            compute(b0, i, end - chunk);
        }
    }
}

template <int GPC, int STYPE, int CT, bool SILU, int ROWS>
__global__ __launch_bounds__(w4g_max_waves(ROWS, CT) * 64) void w4_group_kernel(W4Args p, GroupedRows g,
                                                                            uint32_t col_tiles, uint32_t wave_bytes) {
    static_assert(!SILU || CT == 2, "a gate and an up tile");
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nwaves = blockDim.x >> 6;
    RowTile t = RowTiles(g, ROWS, lane).find(blockIdx.x / col_tiles);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.rows == 0) return;
    constexpr uint32_t kOut = SILU ? 1 : CT;  // output column tiles
    const uint32_t col0 = blockIdx.x % col_tiles * (kOut * kW4gCols);
    v4f acc[CT];
    w4_rows<GPC, STYPE, CT, SILU, ROWS>(p, g, t, col0, smem + wave * wave_bytes, lane, wave, acc);

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
            constexpr float kUp = 1 << kDown;
            float y = acc[ot][r] * kUp;
            if constexpr (SILU) y = y / (1.0f + expf(-y)) * (acc[1][r] * kUp);
            if (row + r < t.rows && col < p.cols)
                p.out[(uint64_t)(t.row0 + row + r) * p.cols + col] = f32_to_bf16_rne(y);
        }
    }
}

template <int STYPE, int CT, bool SILU, int ROWS>
hipError_t launch(const W4Args &p, const GroupedRows &g, uint32_t group, const W4gPlan &plan, hipStream_t s) {
    auto kernel = group == 32    ? w4_group_kernel<4, STYPE, CT, SILU, ROWS>
                  : group == 64  ? w4_group_kernel<2, STYPE, CT, SILU, ROWS>
                  : group == 128 ? w4_group_kernel<1, STYPE, CT, SILU, ROWS>
                                 : w4_group_kernel<0, STYPE, CT, SILU, ROWS>;
    hipLaunchKernelGGL(kernel, dim3(plan.col_tiles * plan.row_tiles), dim3(64 * plan.waves), plan.lds, s, p, g,
                       plan.col_tiles, plan.wave_bytes);
    return hipGetLastError();
}

template <int STYPE>
hipError_t launch_rows(const W4Args &p, const GroupedRows &g, uint32_t group, bool silu, const W4gPlan &plan,
                       hipStream_t s) {
    if (plan.rows == kW4gFew)
        return silu ? launch<STYPE, 2, true, kW4gFew>(p, g, group, plan, s)
                    : launch<STYPE, 1, false, kW4gFew>(p, g, group, plan, s);
    if (silu) return launch<STYPE, 2, true, kW4gRows>(p, g, group, plan, s);
    return plan.ct == 2 ? launch<STYPE, 2, false, kW4gRows>(p, g, group, plan, s)
                        : launch<STYPE, 1, false, kW4gRows>(p, g, group, plan, s);
}

}  // namespace

hipError_t launch_w4_group(const uint16_t *x, const uint8_t *w, const void *scale, int scale_type,
                           const uint8_t *zero, uint32_t group, uint16_t *out, const GroupedRows &g, bool silu,
                           uint32_t n, uint32_t k, hipStream_t s) {
    const uint32_t cols = silu ? n / 2 : n;
    const W4gPlan plan = w4_group_plan(g.rows, g.experts, cols, k, group, silu);
    const W4Args p = {x, w, scale, zero, out, n, k, cols, plan.chunks_per_wave};
    if (scale_type == 0) return launch_rows<0>(p, g, group, silu, plan, s);
    if (scale_type == 1) return launch_rows<1>(p, g, group, silu, plan, s);
    return launch_rows<2>(p, g, group, silu, plan, s);
}

}  // namespace bsr
