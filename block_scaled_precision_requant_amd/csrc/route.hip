// route.hip -- the expert router and the weighted sum back to the tokens.
//
// Router.  For each token the top_k experts by logit, their weights, and the
// stable order of all (token, slot) pairs by expert.  One wave per row: a lane
// holds VPL consecutive logits as order-preserving 32-bit keys, and each of the
// top_k steps is one wave maximum; the lowest lane (hence the lowest index)
// that holds it wins.  Key 0 marks what is never taken (-inf, NaN, behind the
// row's end).  The order is a counting sort without global atomics: every
// block of tokens counts its experts (workspace, [block][expert]), a second
// launch sums the counts of the blocks before it and ranks its own slots 1024
// at a time -- within a wave by ballots over the bits of the expert id, across
// the waves by a prefix over their counts.  Nothing depends on the order in
// which workgroups run.  Few tokens take both steps in one workgroup.
//
// Combine.  out[t] = residual[t] + sum over slots of weight * y[pos]: one pass
// over the routed rows, bound by reading them once.
#include "moe_internal.h"

namespace bsr {
namespace {

__device__ __forceinline__ uint32_t logit_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);  // -0 counts as +0
    if (!(v > -__builtin_huge_valf())) return 0;   // -inf and NaN
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = max(v, (uint32_t)__shfl_xor(v, d));
    return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// Top-k of one row by one wave; lane j < top_k ends with slot j's id (-1:
// none) and weight.
template <int TYPE, int VPL>
__device__ __forceinline__ void select_row(const void *logits, uint64_t row_at, uint32_t experts, uint32_t top_k,
                                           bool sigmoid, bool renorm, float scale, int lane, int32_t &id,
                                           float &weight) {
    uint32_t key[VPL];
    const uint32_t e0 = lane * VPL;
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = e0 + j < experts ? logit_key(load_f32<TYPE>(logits, row_at + e0 + j)) : 0;
    uint32_t all[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) all[j] = key[j];

    id = -1;
    uint32_t taken = 0, top = 0;  // lane j: key of slot j; the row's largest key
    for (uint32_t s = 0; s < top_k; ++s) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int j = 1; j < VPL; ++j)
            if (key[j] > best) {
                best = key[j];
                at = j;
            }
        const uint32_t m = wave_max(best);
        if (m == 0) break;
        const int owner = __builtin_ctzll(__ballot(best == m));
        const int oat = __builtin_amdgcn_readlane(at, owner);
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (lane == owner && j == oat) key[j] = 0;
        if (s == 0) top = m;
        if ((uint32_t)lane == s) {
            id = owner * VPL + oat;
            taken = m;
        }
    }
    const float vmax = top != 0 ? key_logit(top) : 0.0f;
    // exp(v - vmax) with equal infinities at distance 0
    auto rel = [&](uint32_t k) {
        const float v = key_logit(k);
        return k == 0 ? 0.0f : expf(v == vmax ? 0.0f : v - vmax);
    };
    float p;
    if (sigmoid) {
        // 1 / (1 + e^-v) and e^(v - m) / (1 + e^v); a renormalised row of large
        // negative logits keeps its ratios through the common factor e^-m
        const float v = key_logit(taken);
        const float m = renorm ? fminf(vmax, 0.0f) : 0.0f;
        p = taken == 0 ? 0.0f : (v >= 0.0f ? 1.0f / (1.0f + expf(-v)) : expf(v - m) / (1.0f + expf(v)));
    } else {
        p = rel(taken);
    }
    float total = 1.0f;
    if (renorm) {
        total = wave_sum(p);
    } else if (!sigmoid) {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) part += rel(all[j]);
        total = wave_sum(part);
    }
    weight = taken == 0 ? 0.0f : p / total * scale;
}

struct RouteShared {
    uint32_t total[kRouteMaxExperts];               // counts, then first rows, of the experts
    uint32_t before[kRouteMaxExperts];              // of the blocks before this one, then the running row
    uint16_t wave_count[kRouteWaves][kRouteMaxExperts];  // of 64 slots each, then their prefix
    uint32_t wave_sums[kRouteWaves];
};

// total[] -> exclusive prefix over the experts; returns the sum.
__device__ __forceinline__ uint32_t scan_experts(RouteShared &sh, uint32_t experts, int tid) {
    const int lane = tid & 63, wave = tid >> 6;
    const uint32_t v = (uint32_t)tid < experts ? sh.total[tid] : 0;
    uint32_t incl = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) sh.wave_sums[wave] = incl;
    __syncthreads();
    uint32_t base = 0, sum = 0;
    for (int w = 0; w < (int)kRouteWaves; ++w) {
        if (w == wave) base = sum;
        sum += sh.wave_sums[w];
    }
    if ((uint32_t)tid < experts) sh.total[tid] = base + incl - v;
    __syncthreads();
    return sum;
}

// Rows of the slots [s0, s1) of this block; sh.before[e]: the next row of e.
__device__ __forceinline__ void place_slots(RouteShared &sh, const int32_t *ids, int32_t *row_token, int32_t *pos,
                                            uint32_t s0, uint32_t s1, uint32_t experts, uint32_t top_k, int tid) {
    const int lane = tid & 63, wave = tid >> 6;
    const int bits = 32 - __builtin_clz(experts);  // ids 0 .. experts - 1, and `experts` for none
    for (uint32_t base = s0; base < s1; base += kRouteThreads) {
        for (uint32_t e = lane; e < experts; e += 64) sh.wave_count[wave][e] = 0;
        const uint32_t slot = base + tid;
        const int32_t id = slot < s1 ? ids[slot] : -1;
        const uint32_t key = id < 0 ? experts : (uint32_t)id;
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const bool bit = (key >> b) & 1;
            const uint64_t set = __ballot(bit);
            same &= bit ? set : ~set;
        }
        const uint32_t rank = __builtin_popcountll(same & ((1ull << lane) - 1));
        if (id >= 0 && rank == 0) sh.wave_count[wave][id] = (uint16_t)__builtin_popcountll(same);
        __syncthreads();
        uint32_t sum = 0;
        if ((uint32_t)tid < experts)
            for (int w = 0; w < (int)kRouteWaves; ++w) {
                const uint32_t c = sh.wave_count[w][tid];
                sh.wave_count[w][tid] = (uint16_t)sum;
                sum += c;
            }
        __syncthreads();
        if (slot < s1) {
            int32_t row = -1;
            if (id >= 0) {
                row = (int32_t)(sh.before[id] + sh.wave_count[wave][id] + rank);
                row_token[row] = (int32_t)(slot / top_k);
            }
            pos[slot] = row;
        }
        __syncthreads();
        if ((uint32_t)tid < experts) sh.before[tid] += sum;
    }
}

template <int TYPE, int VPL>
__global__ __launch_bounds__(kRouteThreads) void route_select_kernel(
    const void *__restrict__ logits, uint32_t ld, int32_t *ids, float *__restrict__ weights,
    int32_t *__restrict__ offsets, int32_t *__restrict__ row_token, int32_t *__restrict__ pos, uint32_t tokens,
    uint32_t experts, uint32_t top_k, bool sigmoid, bool renorm, float scale, uint32_t *__restrict__ hist,
    uint32_t per_block) {
    __shared__ RouteShared sh;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint32_t t0 = blockIdx.x * per_block, t1 = min(tokens, t0 + per_block);
    if ((uint32_t)tid < experts) {
        sh.total[tid] = 0;
        sh.before[tid] = 0;
    }
    __syncthreads();
    for (uint32_t t = t0 + wave; t < t1; t += kRouteWaves) {
        int32_t id;
        float w;
        select_row<TYPE, VPL>(logits, (uint64_t)t * ld, experts, top_k, sigmoid, renorm, scale, lane, id, w);
        if ((uint32_t)lane < top_k) {
            ids[(uint64_t)t * top_k + lane] = id;
            weights[(uint64_t)t * top_k + lane] = w;
            if (id >= 0) atomicAdd(&sh.total[id], 1u);  // LDS integer counts: any order gives the same
        }
    }
    __syncthreads();
    if (hist != nullptr) {
        if ((uint32_t)tid < experts) hist[(uint64_t)blockIdx.x * experts + tid] = sh.total[tid];
        return;
    }
    const uint32_t sum = scan_experts(sh, experts, tid);
    if ((uint32_t)tid < experts) {
        sh.before[tid] = sh.total[tid];
        offsets[tid] = (int32_t)sh.total[tid];
    }
    if (tid == 0) offsets[experts] = (int32_t)sum;
    __syncthreads();
    place_slots(sh, ids, row_token, pos, 0, tokens * top_k, experts, top_k, tid);
}

__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(
    const int32_t *__restrict__ ids, int32_t *__restrict__ offsets, int32_t *__restrict__ row_token,
    int32_t *__restrict__ pos, uint32_t tokens, uint32_t experts, uint32_t top_k, const uint32_t *__restrict__ hist,
    uint32_t per_block) {
    __shared__ RouteShared sh;
    const int tid = threadIdx.x;
    if ((uint32_t)tid < experts) {
        sh.total[tid] = 0;
        sh.before[tid] = 0;
    }
    __syncthreads();
    // the threads of one expert column share the blocks among them
    uint32_t cols = 64;
    while (cols < experts) cols *= 2;
    const uint32_t e = tid % cols, part = tid / cols, parts = kRouteThreads / cols;
    if (e < experts) {
        uint32_t sum = 0, mine = 0;
        for (uint32_t b = part; b < gridDim.x; b += parts) {
            const uint32_t c = hist[(uint64_t)b * experts + e];
            sum += c;
            if (b < blockIdx.x) mine += c;
        }
        atomicAdd(&sh.total[e], sum);
        atomicAdd(&sh.before[e], mine);
    }
    __syncthreads();
    const uint32_t sum = scan_experts(sh, experts, tid);
    if ((uint32_t)tid < experts) {
        sh.before[tid] += sh.total[tid];
        if (blockIdx.x == 0) offsets[tid] = (int32_t)sh.total[tid];
    }
    if (blockIdx.x == 0 && tid == 0) offsets[experts] = (int32_t)sum;
    __syncthreads();
    const uint32_t t0 = blockIdx.x * per_block, t1 = min(tokens, t0 + per_block);
    place_slots(sh, ids, row_token, pos, t0 * top_k, t1 * top_k, experts, top_k, tid);
}

template <int TYPE>
void launch_select(const void *logits, uint32_t ld, int32_t *ids, float *weights, int32_t *offsets, int32_t *row_token,
                   int32_t *pos, uint32_t tokens, uint32_t experts, uint32_t top_k, bool sigmoid, bool renorm,
                   float scale, uint32_t *hist, const RoutePlan &plan, hipStream_t s) {
    const uint32_t grid = plan.blocks == 0 ? 1 : plan.blocks;
#define BSR_ROUTE(V)                                                                                             \
    hipLaunchKernelGGL((route_select_kernel<TYPE, V>), dim3(grid), dim3(kRouteThreads), 0, s, logits, ld, ids,    \
                       weights, offsets, row_token, pos, tokens, experts, top_k, sigmoid, renorm, scale, hist,    \
                       plan.per_block)
    if (experts <= 64)
        BSR_ROUTE(1);
    else if (experts <= 128)
        BSR_ROUTE(2);
    else if (experts <= 256)
        BSR_ROUTE(4);
    else if (experts <= 512)
        BSR_ROUTE(8);
    else
        BSR_ROUTE(16);
#undef BSR_ROUTE
}

// ---------------------------------------------------------------- combine

constexpr int kCombineThreads = 256;

// V columns per lane (8: 16-byte rows; 1: any n and alignment).
template <int V>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(
    const uint16_t *__restrict__ y, const int32_t *__restrict__ pos, const float *__restrict__ weights,
    const uint16_t *residual, uint16_t *out, uint32_t top_k, uint32_t rows, uint32_t n, uint32_t chunks) {
    typedef uint16_t vec __attribute__((ext_vector_type(V)));
    const uint32_t t = blockIdx.x / chunks;
    const uint64_t c = ((uint64_t)(blockIdx.x % chunks) * kCombineThreads + threadIdx.x) * V;
    if (c >= n) return;
    float acc[V];
    if (residual != nullptr) {
        const vec r = *reinterpret_cast<const vec *>(residual + (uint64_t)t * n + c);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = bf16_to_f32(r[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
    }
    for (uint32_t j = 0; j < top_k; ++j) {
        const uint32_t p = (uint32_t)pos[(uint64_t)t * top_k + j];
        if (p >= rows) continue;  // negative positions too
        const float w = weights[(uint64_t)t * top_k + j];
        const vec v = *reinterpret_cast<const vec *>(y + (uint64_t)p * n + c);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(w, bf16_to_f32(v[i]), acc[i]);
    }
    vec o;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = f32_to_bf16_rne(acc[i]);
    *reinterpret_cast<vec *>(out + (uint64_t)t * n + c) = o;
}

}  // namespace

hipError_t launch_moe_route(const void *logits, int type, uint32_t ld, int32_t *ids, float *weights, int32_t *offsets,
                            int32_t *row_token, int32_t *pos, uint32_t tokens, uint32_t experts, uint32_t top_k,
                            bool sigmoid, bool renorm, float scale, uint32_t *hist, const RoutePlan &plan,
                            hipStream_t s) {
    if (plan.blocks <= 1) hist = nullptr;
    auto select = type == 0 ? launch_select<0> : (type == 1 ? launch_select<1> : launch_select<2>);
    select(logits, ld, ids, weights, offsets, row_token, pos, tokens, experts, top_k, sigmoid, renorm, scale, hist, plan,
           s);
    if (hipError_t e = hipGetLastError()) return e;
    if (hist == nullptr) return hipSuccess;
    hipLaunchKernelGGL(route_place_kernel, dim3(plan.blocks), dim3(kRouteThreads), 0, s, ids, offsets, row_token, pos,
                       tokens, experts, top_k, hist, plan.per_block);
    return hipGetLastError();
}

hipError_t launch_moe_combine(const uint16_t *y, const int32_t *pos, const float *weights, const uint16_t *residual,
                              uint16_t *out, uint32_t tokens, uint32_t top_k, uint32_t rows, uint32_t n,
                              hipStream_t s) {
    const uintptr_t any = reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(residual) |
                          reinterpret_cast<uintptr_t>(out);
    if (n % 8 == 0 && any % 16 == 0) {
        const uint32_t chunks = (uint32_t)div_up(n, 8 * kCombineThreads);
        hipLaunchKernelGGL((combine_kernel<8>), dim3(tokens * chunks), dim3(kCombineThreads), 0, s, y, pos, weights,
                           residual, out, top_k, rows, n, chunks);
    } else {
        const uint32_t chunks = (uint32_t)div_up(n, kCombineThreads);
        hipLaunchKernelGGL((combine_kernel<1>), dim3(tokens * chunks), dim3(kCombineThreads), 0, s, y, pos, weights,
                           residual, out, top_k, rows, n, chunks);
    }
    return hipGetLastError();
}

}  // namespace bsr
