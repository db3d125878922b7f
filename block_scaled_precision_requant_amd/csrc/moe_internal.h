// moe_internal.h -- launchers and device helpers of the expert-layer kernels.
#pragma once

#include "bsr_internal.h"
#include "moe_geometry.h"

namespace bsr {

// Launchers (no validation: the C-ABI layer has checked every argument).
hipError_t launch_moe_route(const void *logits, int type, uint32_t ld, int32_t *ids, float *weights, int32_t *offsets,
                            int32_t *row_token, int32_t *pos, uint32_t tokens, uint32_t experts, uint32_t top_k,
                            bool sigmoid, bool renorm, float scale, uint32_t *hist, const RoutePlan &plan,
                            hipStream_t s);
hipError_t launch_moe_combine(const uint16_t *y, const int32_t *pos, const float *weights, const uint16_t *residual,
                              uint16_t *out, uint32_t tokens, uint32_t top_k, uint32_t rows, uint32_t n,
                              hipStream_t s);
// Columns per lane there: 8 where rows are whole 16-byte words, else 1.
inline uint32_t combine_columns(const uint16_t *y, const uint16_t *residual, const uint16_t *out, uint32_t n) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(residual) |
                          reinterpret_cast<uintptr_t>(out);
    return n % 8 == 0 && any % 16 == 0 ? 8 : 1;
}

// Rows of a grouped call: expert e owns rows [offsets[e], offsets[e + 1]) and
// row p reads operand row index[p] (p where index is null).  offsets null: one
// expert owns all rows.
struct GroupedRows {
    const int32_t *offsets;
    const int32_t *index;
    uint32_t src_rows, rows, experts;

#ifdef __HIPCC__
    // Rows of expert e, empty past the last expert.  The offsets come from the
    // device unchecked: clamped to [0, rows], a descending pair is empty.
    __device__ __forceinline__ void range(uint32_t e, uint32_t &lo, uint32_t &hi) const {
        lo = hi = 0;
        if (e < experts) {
            lo = (uint32_t)min(max(offsets[e], 0), (int32_t)rows);
            hi = (uint32_t)min(max(offsets[e + 1], (int32_t)lo), (int32_t)rows);
        }
    }
#endif
};

hipError_t launch_grouped_gemm(const int8_t *a, const int8_t *w, const float *a_s, const float *w_s, uint16_t *out,
                               const GroupedRows &g, uint32_t n, uint32_t k, hipStream_t s);
// The same for few rows per expert (plan from grouped_gemv_plan).
hipError_t launch_grouped_gemv(const int8_t *a, const int8_t *w, const float *a_s, const float *w_s, uint16_t *out,
                               const GroupedRows &g, uint32_t n, uint32_t k, const GroupedGemvPlan &plan,
                               hipStream_t s);
hipError_t launch_w4_group(const uint16_t *x, const uint8_t *w, const void *scale, int scale_type,
                           const uint8_t *zero, uint32_t group, uint16_t *out, const GroupedRows &g, bool silu,
                           uint32_t n, uint32_t k, hipStream_t s);

#ifdef __HIPCC__
struct RowTile {
    uint32_t expert, row0, rows;  // rows == 0: no such tile
};

// The experts' rows in tiles of bm rows, none across two experts: which rows
// the v-th is.  Every lane of the wave must be active; the result is the same
// in all of them.  A lane holds one of 64 experts at a time.
struct RowTiles {
    GroupedRows g;
    uint32_t bm;
    int lane;
    uint32_t lo, hi, incl, tiles;  // this lane's expert: rows, tiles and their inclusive prefix

    __device__ __forceinline__ RowTiles(const GroupedRows &g_, uint32_t bm_, int lane_) : g(g_), bm(bm_), lane(lane_) {
        if (g.offsets != nullptr) load(0);
    }
    __device__ __forceinline__ void load(uint32_t e0) {
        g.range(e0 + lane, lo, hi);
        tiles = (hi - lo + bm - 1) / bm;
        incl = tiles;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
    }
    __device__ __forceinline__ RowTile find(uint32_t v) {
        if (g.offsets == nullptr) {
            const uint32_t row0 = v * bm;
            return {0, row0, row0 < g.rows ? min(bm, g.rows - row0) : 0};
        }
        for (uint32_t e0 = 0;;) {
            const uint64_t past = __ballot(incl > v);
            if (past != 0) {
                const int owner = __builtin_ctzll(past);
                const uint32_t first = __builtin_amdgcn_readlane(incl - tiles, owner);
                const uint32_t olo = __builtin_amdgcn_readlane(lo, owner), ohi = __builtin_amdgcn_readlane(hi, owner);
                const uint32_t row0 = olo + (v - first) * bm;
                return {e0 + owner, row0, min(bm, ohi - row0)};
            }
            v -= __builtin_amdgcn_readlane(incl, 63);
            e0 += 64;
            if (e0 >= g.experts) return {0, 0, 0};
            load(e0);
        }
    }
};

// ---- streamed weights (the two GEMVs) ----
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));

// Lane (c, q) holds dword j of quarter q in component j -> dword q of quarter j:
// a 4 x 4 transposition over the four rows of 16 lanes.
__device__ __forceinline__ v4i swap_quarters(v4i w) {
    const auto a = __builtin_amdgcn_permlane16_swap((uint32_t)w.x, (uint32_t)w.y, false, false);
    const auto b = __builtin_amdgcn_permlane16_swap((uint32_t)w.z, (uint32_t)w.w, false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
    return v4i{(int)c[0], (int)d[0], (int)c[1], (int)d[1]};
}

constexpr int kRsrcWord3 = 0x00020000;         // raw buffer (gfx9)
constexpr uint32_t kPastEnd = 0xFFFFFFE0u;     // an offset behind every buffer: reads as 0

__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t r, uint32_t lane_offset, uint32_t offset) {
    return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(r, lane_offset, offset, 0));
}

// Operand row of output row p, or -1 for a row of zeros.
__device__ __forceinline__ int32_t source_row(const GroupedRows &g, uint32_t p) {
    if (g.index == nullptr) return (int32_t)p;
    const int32_t i = g.index[p];
    return (uint32_t)i < g.src_rows ? i : -1;
}

// An element of `type` (enum bsr_type) as binary32 (exact).
template <int TYPE>
__device__ __forceinline__ float load_f32(const void *p, uint64_t i) {
    if constexpr (TYPE == 0) return __uint_as_float((uint32_t) static_cast<const uint16_t *>(p)[i] << 16);
    if constexpr (TYPE == 1) return (float)static_cast<const _Float16 *>(p)[i];
    return static_cast<const float *>(p)[i];
}
__device__ __forceinline__ float bf16_to_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
#endif

}  // namespace bsr
