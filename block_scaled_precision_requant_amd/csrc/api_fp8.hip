// api_fp8.hip -- the C ABI of the FP8 products, their weight quantizer and the
// operators around sorted tokens: argument validation and the launches, under the
// same rules as api.hip (every check before the first launch, nothing kept between
// calls).
#include "api_common.h"
#include "bsr.h"
#include "fp8_internal.h"

using bsr::aligned;
using bsr::check_device;
using bsr::div_up;
using bsr::fp8_k_ok;
using bsr::kFp8Block;
using bsr::kMaxThreads;
using bsr::launched;

namespace {

constexpr uint32_t kMaxExperts = 65536;
constexpr uint64_t kMaxRows = (1ull << 31) - 1;

int product_check(const void *a_q, const void *w_q, const float *a_scale, const float *w_scale, const uint16_t *out) {
    if (!a_q || !w_q || !a_scale || !w_scale || !out) return BSR_ENULL;
    if (!aligned(a_q, 16) || !aligned(w_q, 16) || !aligned(a_scale, 4) || !aligned(w_scale, 4) || !aligned(out, 2))
        return BSR_EALIGN;
    return BSR_OK;
}

int product(const bsr::Fp8Args &p, void *stream) {
    if (bsr::fp8_choice(p.rows.rows, p.rows.experts, p.n, p.k, p.silu).threads > kMaxThreads)
        return BSR_EINVAL;
    if (int st = check_device()) return st;
    return launched(bsr::launch_fp8_gemm(p, static_cast<hipStream_t>(stream)));
}

// Rows of tokens: sizes, and one workgroup per chunk of a token's row or per slot.
bool tokens_ok(uint32_t tokens, uint32_t top_k, uint32_t n) {
    return top_k != 0 && top_k <= bsr::kRouteMaxTopK && n <= kMaxRows &&
           tokens * div_up(n, 8 * bsr::kTokenThreads) * bsr::kTokenThreads <= kMaxThreads &&
           (uint64_t)tokens * top_k * bsr::kTokenThreads <= kMaxThreads;
}

}  // namespace

extern "C" {

int quantize_w_fp8(const uint16_t *w_bf16, uint8_t *w_q, float *w_scale, uint8_t *w_qt, float *w_scale_t,
                   uint32_t experts, uint32_t n, uint32_t k, void *stream) {
    if (k == 0 || k % kFp8Block != 0) return BSR_EINVAL;
    if (w_qt != nullptr && n % kFp8Block != 0) return BSR_EINVAL;
    if (experts == 0 || n == 0) return BSR_OK;
    if (!w_bf16 || !w_q || !w_scale || (w_qt == nullptr) != (w_scale_t == nullptr)) return BSR_ENULL;
    if (!aligned(w_bf16, 16) || !aligned(w_q, 16) || !aligned(w_scale, 4) || !aligned(w_qt, 16) || !aligned(w_scale_t, 4))
        return BSR_EALIGN;
    const uint64_t blocks = div_up(n, kFp8Block) * (k / kFp8Block);  // (below 2^50: of all experts it may pass 64 bits)
    if (blocks > kMaxThreads / bsr::kQwThreads / experts) return BSR_EINVAL;
    if (int st = check_device()) return st;
    return launched(bsr::launch_quantize_w_fp8(w_bf16, w_q, w_scale, w_qt, w_scale_t, experts, n, k,
                                               static_cast<hipStream_t>(stream)));
}

int fp8_gemm_blockscaled(const uint8_t *a_q, const uint8_t *w_q, const float *a_scale, const float *w_scale,
                         uint16_t *out, uint32_t m, uint32_t n, uint32_t k, void *stream) {
    if (!fp8_k_ok(k) || m > kMaxRows || n > kMaxRows) return BSR_EINVAL;
    if (m == 0 || n == 0) return BSR_OK;
    if (int st = product_check(a_q, w_q, a_scale, w_scale, out)) return st;
    return product({a_q, w_q, a_scale, w_scale, out, {nullptr, nullptr, m, m, 1}, n, k, false}, stream);
}

int fp8_grouped_gemm_blockscaled(const uint8_t *a_q, const uint8_t *w_q, const float *a_scale, const float *w_scale,
                                 const int32_t *offsets, const int32_t *row_index, int silu_mul, uint16_t *out,
                                 uint32_t a_rows, uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, void *stream) {
    if (!fp8_k_ok(k) || rows > kMaxRows || n > kMaxRows || experts > kMaxExperts) return BSR_EINVAL;
    if ((silu_mul != 0 && silu_mul != 1) || (silu_mul == 1 && n % (2 * kFp8Block) != 0)) return BSR_EINVAL;
    if (row_index != nullptr ? a_rows == 0 && rows != 0 : a_rows < rows) return BSR_EINVAL;
    if (row_index != nullptr && (uint64_t)a_rows * k >= (1ull << 32)) return BSR_EINVAL;
    if (rows == 0 || n == 0 || experts == 0) return BSR_OK;
    if (!offsets) return BSR_ENULL;
    if (int st = product_check(a_q, w_q, a_scale, w_scale, out)) return st;
    if (!aligned(offsets, 4) || !aligned(row_index, 4)) return BSR_EALIGN;
    return product({a_q, w_q, a_scale, w_scale, out, {offsets, row_index, a_rows, rows, experts}, n, k, silu_mul == 1},
                   stream);
}

int moe_dispatch(const uint16_t *x, const int32_t *pos, uint16_t *out, uint32_t tokens, uint32_t top_k, uint32_t rows,
                 uint32_t n, void *stream) {
    if (!tokens_ok(tokens, top_k, n)) return BSR_EINVAL;
    if (tokens == 0 || n == 0) return BSR_OK;
    if (!x || !pos || (rows != 0 && !out)) return BSR_ENULL;
    if (!aligned(x, 2) || !aligned(pos, 4) || !aligned(out, 2)) return BSR_EALIGN;
    if (int st = check_device()) return st;
    return launched(bsr::launch_moe_dispatch(x, pos, out, tokens, top_k, rows, n, static_cast<hipStream_t>(stream)));
}

int moe_dispatch_grad(const uint16_t *d_rows, const int32_t *pos, uint16_t *d_x, uint32_t tokens, uint32_t top_k,
                      uint32_t rows, uint32_t n, void *stream) {
    if (!tokens_ok(tokens, top_k, n)) return BSR_EINVAL;
    if (tokens == 0 || n == 0) return BSR_OK;
    if ((rows != 0 && !d_rows) || !pos || !d_x) return BSR_ENULL;
    if (!aligned(d_rows, 2) || !aligned(pos, 4) || !aligned(d_x, 2)) return BSR_EALIGN;
    if (int st = check_device()) return st;
    return launched(bsr::launch_moe_dispatch_grad(d_rows, pos, d_x, tokens, top_k, rows, n,
                                                  static_cast<hipStream_t>(stream)));
}

int moe_combine_grad(const uint16_t *d_out, const uint16_t *y, const int32_t *pos, const float *weights, uint16_t *d_y,
                     float *d_weights, uint32_t tokens, uint32_t top_k, uint32_t rows, uint32_t n, void *stream) {
    if (!tokens_ok(tokens, top_k, n)) return BSR_EINVAL;
    if (tokens == 0) return BSR_OK;
    if ((n != 0 && !d_out) || (rows != 0 && n != 0 && (!y || !d_y)) || !pos || !weights || !d_weights) return BSR_ENULL;
    if (!aligned(d_out, 2) || !aligned(y, 2) || !aligned(pos, 4) || !aligned(weights, 4) || !aligned(d_y, 2) ||
        !aligned(d_weights, 4))
        return BSR_EALIGN;
    if (int st = check_device()) return st;
    return launched(bsr::launch_moe_combine_grad(d_out, y, pos, weights, d_y, d_weights, tokens, top_k, rows, n,
                                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
