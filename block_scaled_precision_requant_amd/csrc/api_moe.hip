// api_moe.hip -- the C ABI of the expert-layer operators: argument validation
// and the launches, under the same rules as api.hip (every check before the
// first launch, nothing kept between calls).
#include <cmath>

#include "api_common.h"
#include "bsr.h"
#include "moe_internal.h"

using bsr::aligned;
using bsr::check_device;
using bsr::div_up;
using bsr::k_ok;
using bsr::kMaxGrid;
using bsr::kMaxThreads;
using bsr::launched;

namespace {

constexpr uint32_t kMaxExperts = 65536;
constexpr uint64_t kMaxRows = (1ull << 31) - 1;

uintptr_t type_bytes(int type) { return type == BSR_TYPE_F32 ? 4 : 2; }
bool type_ok(int type) { return type == BSR_TYPE_BF16 || type == BSR_TYPE_F16 || type == BSR_TYPE_F32; }

// Shapes the grouped calls share; `src_rows` operand rows.
bool grouped_ok(const int32_t *row_index, uint32_t src_rows, uint32_t rows, uint32_t experts) {
    return rows <= kMaxRows && experts <= kMaxExperts &&
           (row_index != nullptr ? src_rows != 0 || rows == 0 : src_rows >= rows);
}

int w4_check(const uint16_t *x, const uint8_t *w_packed, const void *scale, int scale_type, const uint16_t *out) {
    if (!x || !w_packed || !scale || !out) return BSR_ENULL;
    if (!aligned(x, 16) || !aligned(w_packed, 16) || !aligned(scale, type_bytes(scale_type)) || !aligned(out, 2))
        return BSR_EALIGN;
    return BSR_OK;
}

bool w4_shape_ok(int scale_type, uint32_t group, uint32_t x_rows, uint32_t k) {
    return k_ok(k) && k < bsr::kGemmTallMaxK && (uint64_t)x_rows * k < (1ull << 31) && type_ok(scale_type) &&
           (group == 0 || ((group == 32 || group == 64 || group == 128) && k % group == 0));
}

bool w4_grid_ok(uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, uint32_t group, bool silu) {
    return bsr::grouped_row_tiles(rows, experts, 16) * div_up(n, 16) <= kMaxGrid &&
           bsr::w4_group_threads(bsr::w4_group_plan(rows, experts, silu ? n / 2 : n, k, group, silu)) <= kMaxThreads;
}

}  // namespace

extern "C" {

uint64_t moe_route_ws_bytes(uint32_t tokens, uint32_t experts, uint32_t top_k) {
    (void)top_k;
    if (experts == 0 || experts > bsr::kRouteMaxExperts) return 0;  // moe_route refuses these
    return bsr::moe_route_plan(tokens, experts).bytes;
}

int moe_route(const void *logits, int type, uint32_t ld, int32_t *ids, float *weights, int32_t *offsets,
              int32_t *row_token, int32_t *pos, uint32_t tokens, uint32_t experts, uint32_t top_k, int score,
              int renorm, float scale, void *workspace, uint64_t workspace_bytes, void *stream) {
    if (!type_ok(type) || (score != BSR_SCORE_SOFTMAX && score != BSR_SCORE_SIGMOID) || !std::isfinite(scale))
        return BSR_EINVAL;
    if (experts == 0 || experts > bsr::kRouteMaxExperts || ld < experts) return BSR_EINVAL;
    if (top_k == 0 || top_k > experts || top_k > bsr::kRouteMaxTopK) return BSR_EINVAL;
    if ((uint64_t)tokens * top_k > kMaxRows) return BSR_EINVAL;
    if (!offsets) return BSR_ENULL;
    if (tokens != 0 && (!logits || !ids || !weights || !row_token || !pos)) return BSR_ENULL;
    if (!aligned(logits, type_bytes(type)) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(offsets, 4) ||
        !aligned(row_token, 4) || !aligned(pos, 4))
        return BSR_EALIGN;
    const bsr::RoutePlan plan = bsr::moe_route_plan(tokens, experts);
    if (plan.bytes != 0) {
        if (!workspace) return BSR_ENULL;
        if (!aligned(workspace, 16)) return BSR_EALIGN;
        if (workspace_bytes < plan.bytes) return BSR_EINVAL;
    }
    if (int st = check_device()) return st;
    return launched(bsr::launch_moe_route(logits, type, ld, ids, weights, offsets, row_token, pos, tokens, experts,
                                          top_k, score == BSR_SCORE_SIGMOID, renorm != 0, scale,
                                          static_cast<uint32_t *>(workspace), plan,
                                          static_cast<hipStream_t>(stream)));
}

int int8_grouped_gemm_blockscaled(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale, const float *w_scale,
                                  const int32_t *offsets, const int32_t *row_index, uint16_t *out, uint32_t a_rows,
                                  uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, void *stream) {
    if (!k_ok(k) || k >= bsr::kGemmTallMaxK || !grouped_ok(row_index, a_rows, rows, experts)) return BSR_EINVAL;
    if (row_index != nullptr && (uint64_t)a_rows * k >= (1ull << 32)) return BSR_EINVAL;
    if (rows == 0 || n == 0 || experts == 0) return BSR_OK;
    if (!a_i8 || !w_i8 || !a_scale || !w_scale || !offsets || !out) return BSR_ENULL;
    if (!aligned(a_i8, 16) || !aligned(w_i8, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) ||
        !aligned(offsets, 4) || !aligned(row_index, 4) || !aligned(out, 2))
        return BSR_EALIGN;
    if (bsr::grouped_row_tiles(rows, experts, 16) * div_up(n, 16) > kMaxGrid ||
        bsr::grouped_threads(rows, experts, n, k) > kMaxThreads)
        return BSR_EINVAL;
    if (int st = check_device()) return st;
    return launched(bsr::launch_grouped_gemm(a_i8, w_i8, a_scale, w_scale, out,
                                             {offsets, row_index, a_rows, rows, experts}, n, k,
                                             static_cast<hipStream_t>(stream)));
}

int moe_combine(const uint16_t *y, const int32_t *pos, const float *weights, const uint16_t *residual, uint16_t *out,
                uint32_t tokens, uint32_t top_k, uint32_t rows, uint32_t n, void *stream) {
    if (top_k == 0 || top_k > bsr::kRouteMaxTopK) return BSR_EINVAL;
    if (tokens == 0 || n == 0) return BSR_OK;
    if ((rows != 0 && !y) || !pos || !weights || !out) return BSR_ENULL;
    if (!aligned(y, 2) || !aligned(pos, 4) || !aligned(weights, 4) || !aligned(residual, 2) || !aligned(out, 2))
        return BSR_EALIGN;
    const uint64_t columns = (uint64_t)bsr::combine_columns(y, residual, out, n) * bsr::kCombineThreads;
    if (tokens * div_up(n, columns) * bsr::kCombineThreads > kMaxThreads) return BSR_EINVAL;
    if (int st = check_device()) return st;
    return launched(bsr::launch_moe_combine(y, pos, weights, residual, out, tokens, top_k, rows, n,
                                            static_cast<hipStream_t>(stream)));
}

int w4a16_group_gemv(const uint16_t *x, const uint8_t *w_packed, const void *scale, int scale_type,
                     const uint8_t *zero, uint32_t group, uint16_t *out, uint32_t m, uint32_t n, uint32_t k,
                     void *stream) {
    if (!w4_shape_ok(scale_type, group, m, k)) return BSR_EINVAL;
    if (m == 0 || n == 0) return BSR_OK;
    if (int st = w4_check(x, w_packed, scale, scale_type, out)) return st;
    if (!w4_grid_ok(m, 1, n, k, group, false)) return BSR_EINVAL;
    if (int st = check_device()) return st;
    return launched(bsr::launch_w4_group(x, w_packed, scale, scale_type, zero, group, out,
                                         {nullptr, nullptr, m, m, 1}, false, n, k, static_cast<hipStream_t>(stream)));
}

int w4a16_group_gemv_experts(const uint16_t *x, const uint8_t *w_packed, const void *scale, int scale_type,
                             const uint8_t *zero, uint32_t group, const int32_t *offsets, const int32_t *row_index,
                             int silu_mul, uint16_t *out, uint32_t x_rows, uint32_t rows, uint32_t experts, uint32_t n,
                             uint32_t k, void *stream) {
    if (!w4_shape_ok(scale_type, group, x_rows, k) || !grouped_ok(row_index, x_rows, rows, experts)) return BSR_EINVAL;
    if ((silu_mul != 0 && silu_mul != 1) || (silu_mul == 1 && n % 2 != 0)) return BSR_EINVAL;
    if (rows == 0 || n == 0 || experts == 0) return BSR_OK;
    if (!offsets) return BSR_ENULL;
    if (int st = w4_check(x, w_packed, scale, scale_type, out)) return st;
    if (!aligned(offsets, 4) || !aligned(row_index, 4)) return BSR_EALIGN;
    if (!w4_grid_ok(rows, experts, n, k, group, silu_mul == 1)) return BSR_EINVAL;
    if (int st = check_device()) return st;
    return launched(bsr::launch_w4_group(x, w_packed, scale, scale_type, zero, group, out,
                                         {offsets, row_index, x_rows, rows, experts}, silu_mul == 1, n, k,
                                         static_cast<hipStream_t>(stream)));
}

}  // extern "C"
