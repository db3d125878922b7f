// moe_tokens.hip -- rows of tokens copied into the experts' order, the gradient of
// that copy, and the gradient of the weighted sum that brings rows back (combine, in
// route.hip).
//
//   dispatch       out[pos[t,s]] = x[t]
//   its gradient   d_x[t] = sum_s d_rows[pos[t,s]]
//   of combine     d_y[pos[t,s]] = weights[t,s] * d_out[t]
//                  d_weights[t,s] = sum_j d_out[t,j] * y[pos[t,s],j]
//
// All walk the tokens: a token's row is read once (dispatch, combine's gradient) or
// written once, and each of its routed rows is read or written once, in runs of 16
// bytes a lane.  Slots whose position is outside the rows are skipped.  Bound by HBM
// (a device copy of 1 GiB: 5.1 TB/s).  MI355X, 8192 tokens, top 8, n 4096: dispatch's
// gradient 116 us, 5.2 TB/s; combine's 211, 5.4.  777 tokens, top 6, n 4095, rows at odd
// alignments: dispatch 9.1 us, 4.9 TB/s.
#include "fp8_internal.h"

namespace bsr {
namespace {

__global__ __launch_bounds__(kTokenThreads) void dispatch_kernel(const uint16_t *__restrict__ x,
                                                                 const int32_t *__restrict__ pos,
                                                                 uint16_t *__restrict__ out, uint32_t top_k,
                                                                 uint32_t rows, uint32_t n, uint32_t chunks) {
    const uint32_t t = blockIdx.x / chunks;
    const uint32_t c = (blockIdx.x % chunks * kTokenThreads + threadIdx.x) * 8;
    if (c >= n) return;
    const u16x8 v = load8(x + (uint64_t)t * n, c, n);
    for (uint32_t j = 0; j < top_k; ++j) {
        const uint32_t p = (uint32_t)pos[(uint64_t)t * top_k + j];
        if (p < rows) store8(out + (uint64_t)p * n, c, n, v);  // (negative positions are past the rows too)
    }
}

__global__ __launch_bounds__(kTokenThreads) void dispatch_grad_kernel(const uint16_t *__restrict__ d_rows,
                                                                      const int32_t *__restrict__ pos,
                                                                      uint16_t *__restrict__ d_x, uint32_t top_k,
                                                                      uint32_t rows, uint32_t n, uint32_t chunks) {
    const uint32_t t = blockIdx.x / chunks;
    const uint32_t c = (blockIdx.x % chunks * kTokenThreads + threadIdx.x) * 8;
    if (c >= n) return;
    float acc[8] = {};
    for (uint32_t j = 0; j < top_k; ++j) {
        const uint32_t p = (uint32_t)pos[(uint64_t)t * top_k + j];
        if (p >= rows) continue;
        const u16x8 v = load8(d_rows + (uint64_t)p * n, c, n);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += bf16_to_f32(v[i]);
    }
    u16x8 o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = f32_to_bf16(acc[i]);
    store8(d_x + (uint64_t)t * n, c, n, o);
}

// One workgroup per (token, slot): both sums of a lane go on over the columns, and
// the waves' are added in wave order.
__global__ __launch_bounds__(kTokenThreads) void combine_grad_kernel(
    const uint16_t *__restrict__ d_out, const uint16_t *y, const int32_t *__restrict__ pos,
    const float *__restrict__ weights, uint16_t *d_y, float *__restrict__ d_weights, uint32_t top_k,
    uint32_t rows, uint32_t n) {
    __shared__ float sums[kTokenThreads / 64];
    // all slots of a token on one XCD, whose L2 reads the token's row once (8192 tokens,
    // top 8, n 4096: 211 us; slots in the order of the grid, each on another XCD, 229)
    const uint32_t wg = blockIdx.x, step = kXcds * top_k;
    uint32_t slot = wg;
    if (wg < gridDim.x / step * step) {
        const uint32_t j = wg / kXcds;
        slot = (j / top_k * kXcds + wg % kXcds) * top_k + j % top_k;
    }
    const uint32_t t = slot / top_k;
    const uint32_t p = (uint32_t)pos[slot];
    if (p >= rows) {
        if (threadIdx.x == 0) d_weights[slot] = 0.0f;
        return;
    }
    const float w = weights[slot];
    const uint16_t *dr = d_out + (uint64_t)t * n, *yr = y + (uint64_t)p * n;
    uint16_t *o = d_y + (uint64_t)p * n;
    float sum = 0.0f;
    for (uint32_t c = threadIdx.x * 8; c < n; c += kTokenThreads * 8) {
        const u16x8 d = load8(dr, c, n), v = load8(yr, c, n);
        u16x8 r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = bf16_to_f32(d[i]);
            sum = fmaf(f, bf16_to_f32(v[i]), sum);
            r[i] = f32_to_bf16(w * f);
        }
        store8(o, c, n, r);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
    if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        float total = sums[0];
#pragma unroll
        for (uint32_t i = 1; i < kTokenThreads / 64; ++i) total += sums[i];
        d_weights[slot] = total;
    }
}

uint32_t row_chunks(uint32_t n) { return (uint32_t)div_up(n, 8 * kTokenThreads); }

}  // namespace

hipError_t launch_moe_dispatch(const uint16_t *x, const int32_t *pos, uint16_t *out, uint32_t tokens, uint32_t top_k,
                               uint32_t rows, uint32_t n, hipStream_t s) {
    const uint32_t chunks = row_chunks(n);
    hipLaunchKernelGGL(dispatch_kernel, dim3(tokens * chunks), dim3(kTokenThreads), 0, s, x, pos, out, top_k, rows, n, chunks);
    return hipGetLastError();
}

hipError_t launch_moe_dispatch_grad(const uint16_t *d_rows, const int32_t *pos, uint16_t *d_x, uint32_t tokens,
                                    uint32_t top_k, uint32_t rows, uint32_t n, hipStream_t s) {
    const uint32_t chunks = row_chunks(n);
    hipLaunchKernelGGL(dispatch_grad_kernel, dim3(tokens * chunks), dim3(kTokenThreads), 0, s, d_rows, pos, d_x, top_k, rows,
                       n, chunks);
    return hipGetLastError();
}

hipError_t launch_moe_combine_grad(const uint16_t *d_out, const uint16_t *y, const int32_t *pos, const float *weights,
                                   uint16_t *d_y, float *d_weights, uint32_t tokens, uint32_t top_k, uint32_t rows,
                                   uint32_t n, hipStream_t s) {
    hipLaunchKernelGGL(combine_grad_kernel, dim3(tokens * top_k), dim3(kTokenThreads), 0, s, d_out, y, pos, weights, d_y,
                       d_weights, top_k, rows, n);
    return hipGetLastError();
}

}  // namespace bsr
