// route.hip -- the expert router and the weighted sum back to the tokens.
//
// Router.  For each token the top_k experts by logit, their weights, and the
// stable order of all (token, slot) pairs by expert.  A row takes 16, 32 or 64
// lanes (up to four rows per wave): a lane holds VPL consecutive logits as
// order-preserving 32-bit keys, sorted once, and each of the top_k steps is one
// maximum over the lanes' first keys; the lowest lane (hence the lowest index)
// that holds it wins and moves on to its next.  Key 0 marks what is never taken
// (-inf, NaN, behind the row's end).  The order is a counting sort without global atomics: every
// block of tokens counts its experts (workspace, [block][expert]), a second
// launch sums the counts of the blocks before it and ranks its own slots 1024
// at a time -- within a wave by ballots over the bits of the expert id, across
// the waves by a prefix over their counts.  Nothing depends on the order in
// which workgroups run.  Few tokens take both steps in one workgroup.
//
// MI355X: one token of 64 experts 4.9 us in a graph (an empty launch 3.2); 16384 tokens
// of 256 experts, top 8 (18.9 MB) 21 us: selection 13-15, bound by vector issue (28
// exchanges of the sort and eight maxima per row pair: 6240 vector instructions a SIMD,
// 87 % of the waves' time), order 8, of which the waves wait 54 %: each of the 256
// workgroups reads the whole table of 256 x 256 counts, 64 MB from L2 in all.
//
// Combine.  out[t] = residual[t] + sum over slots of weight * y[pos]: one pass
// over the routed rows, bound by reading them once: 4099 tokens, top 8, n 4096 (301 MB)
// 61 us, 5.0 TB/s (n 4095, a column per lane, 166 us).
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

// Reductions over segments of L = 16, 32 or 64 lanes, the result in every lane:
// rotations within the rows of 16, then swaps of rows.
template <int N>
__device__ __forceinline__ uint32_t row_ror(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xF, 0xF, false);
}
template <int L, class F>
__device__ __forceinline__ uint32_t segment_reduce(uint32_t v, F f) {
    v = f(v, row_ror<8>(v));
    v = f(v, row_ror<4>(v));
    v = f(v, row_ror<2>(v));
    v = f(v, row_ror<1>(v));
    if constexpr (L >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        v = f(p[0], p[1]);
    }
    if constexpr (L >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        v = f(p[0], p[1]);
    }
    return v;
}
template <int L>
__device__ __forceinline__ uint32_t segment_max(uint32_t v) {
    return segment_reduce<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L>
__device__ __forceinline__ float segment_sum(float v) {
    return __uint_as_float(segment_reduce<L>(
        __float_as_uint(v), [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); }));
}

// e^x for x <= 0 (below -200: 0), to about 2 ulp: 2^(x log2 e) with the rounding
// of the product made good to first order; results under 2^-126 may be 0.
__device__ __forceinline__ float exp_neg(float x) {
    x = fmaxf(x, -200.0f);
    const float t = x * 0x1.715476p+0f;
    const float r = fmaf(x, 0x1.715476p+0f, -t) + x * 0x1.4ae0cp-26f;
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * 0x1.62e43p-1f, e);
}

// VPL consecutive logits from element e of a row of `experts` (aligned to the
// element only); those past the end read as -inf.
template <int TYPE, int VPL>
__device__ __forceinline__ void load_logits(const void *logits, uint64_t row_at, uint32_t e, uint32_t experts,
                                            float (&v)[VPL]) {
    if constexpr (TYPE == 2) {
        typedef float f4 __attribute__((ext_vector_type(4), aligned(4)));
        if (e + VPL <= experts) {
#pragma unroll
            for (int j = 0; j < VPL; j += 4) {
                const f4 x = *reinterpret_cast<const f4 *>(static_cast<const float *>(logits) + row_at + e + j);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[j + i] = x[i];
            }
            return;
        }
    } else {
        typedef uint16_t h4 __attribute__((ext_vector_type(4), aligned(2)));
        if (e + VPL <= experts) {
#pragma unroll
            for (int j = 0; j < VPL; j += 4) {
                const h4 x = *reinterpret_cast<const h4 *>(static_cast<const uint16_t *>(logits) + row_at + e + j);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    v[j + i] = TYPE == 0 ? bf16_to_f32(x[i]) : (float)__builtin_bit_cast(_Float16, (uint16_t)x[i]);
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
        v[j] = e + j < experts ? load_f32<TYPE>(logits, row_at + e + j) : -__builtin_huge_valf();
}

// Top-k of one row by a segment of L lanes, VPL consecutive experts each (v: this
// lane's logits); slots: top_k words of LDS of this row.  Lane j < top_k of the
// segment returns slot j's id (-1: none) and weight.
template <int VPL, int L>
__device__ __forceinline__ int32_t select_row(const float (&v)[VPL], uint32_t *slots, uint32_t top_k, bool sigmoid,
                                              bool renorm, float scale, int lane, float &weight) {
    const uint32_t sl = lane % L;  // lane within the segment
    uint32_t key[VPL], all[VPL];
    uint32_t id[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        key[j] = all[j] = logit_key(v[j]);
        id[j] = sl * VPL + j;
    }
    // this lane's experts in falling order, equal ones by index
#pragma unroll
    for (int n = VPL - 1; n > 0; --n)
#pragma unroll
        for (int j = 0; j < n; ++j) {
            // (masks, not selects: a select between two elements would make the index dynamic)
            const uint32_t a = key[j], b = key[j + 1];
            const uint32_t d = (id[j] ^ id[j + 1]) & (b > a ? ~0u : 0u);
            key[j] = max(a, b);
            key[j + 1] = min(a, b);
            id[j] ^= d;
            id[j + 1] ^= d;
        }
    uint32_t taken = 0, top = 0;  // lane j: key of slot j; the row's largest key
    for (uint32_t s = 0; s < top_k; ++s) {
        const uint32_t m = segment_max<L>(key[0]);
        const uint64_t have = __ballot(m != 0 && key[0] == m);
        if (have == 0) break;  // no segment has an expert left
        bool won;
        if constexpr (L == 64)
            won = lane == __builtin_ctzll(have);
        else
            won = (have >> (lane & ~(L - 1)) & ((1ull << L) - 1) & ((2ull << sl) - 1)) == 1ull << sl;
        if (s == 0) top = m;
        if (sl == s) taken = m;
        if (won) {
            slots[s] = id[0];
#pragma unroll
            for (int j = 0; j + 1 < VPL; ++j) {
                key[j] = key[j + 1];
                id[j] = id[j + 1];
            }
            key[VPL - 1] = 0;
        }
    }
    const float vmax = top != 0 ? key_logit(top) : 0.0f;
    // exp(v - vmax) with equal infinities at distance 0
    auto rel = [&](uint32_t k) {
        const float x = key_logit(k);
        return k == 0 ? 0.0f : exp_neg(x == vmax ? 0.0f : x - vmax);
    };
    float p;
    if (sigmoid) {
        // 1 / (1 + e^-v), or e^(v - m) / (1 + e^v) below 0; a renormalised row of large
        // negative logits keeps its ratios through the common factor e^-m
        const float x = key_logit(taken);
        const float m = renorm ? fminf(vmax, 0.0f) : 0.0f;
        p = taken == 0 ? 0.0f : (x >= 0.0f ? 1.0f : exp_neg(x - m)) / (1.0f + exp_neg(-fabsf(x)));
    } else {
        p = rel(taken);
    }
    float total = 1.0f;
    if (renorm) {
        total = segment_sum<L>(p);
    } else if (!sigmoid) {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) part += rel(all[j]);
        total = segment_sum<L>(part);
    }
    weight = taken == 0 ? 0.0f : p / total * scale;
    return taken == 0 ? -1 : (int32_t)slots[sl];
}

struct RouteShared {
    uint32_t total[kRouteMaxExperts];               // counts, then first rows, of the experts
    uint32_t before[kRouteMaxExperts];              // of the blocks before this one, then the running row
    uint16_t wave_count[kRouteWaves][kRouteMaxExperts];  // of 64 slots each, then their prefix
    uint32_t wave_sums[kRouteWaves];
    uint32_t slots[kRouteWaves][4][kRouteMaxTopK];  // ids of the rows that a wave works on
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

template <int TYPE, int VPL, int L>
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
    // a row's logits are asked for while the row before it is worked on
    constexpr uint32_t kRowsPerWave = 64 / L, kStep = kRouteWaves * kRowsPerWave;
    const uint32_t e0 = lane % L * VPL;
    uint32_t t = t0 + wave * kRowsPerWave + lane / L;
    float next[VPL];
    load_logits<TYPE, VPL>(logits, (uint64_t)t * ld, t < t1 ? e0 : experts, experts, next);
    for (uint32_t tw = t0 + wave * kRowsPerWave; tw < t1; tw += kStep, t += kStep) {
        float v[VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) v[j] = next[j];
        load_logits<TYPE, VPL>(logits, (uint64_t)(t + kStep) * ld, t + kStep < t1 ? e0 : experts, experts, next);
        const bool live = t < t1;
        const uint32_t sl = lane % L;
        float weight;
        const int32_t id = select_row<VPL, L>(v, sh.slots[wave][lane / L], top_k, sigmoid, renorm, scale, lane, weight);
        if (live && sl < top_k) {
            ids[(uint64_t)t * top_k + sl] = id;
            weights[(uint64_t)t * top_k + sl] = weight;
            if (id >= 0) atomicAdd(&sh.total[id], 1u);  // LDS integer counts: any order gives the same
        }
    }
    __syncthreads();
    if (hist != nullptr) {
        if ((uint32_t)tid < experts) hist[(uint64_t)blockIdx.x * route_pitch(experts) + tid] = sh.total[tid];
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
    // a thread adds up four experts over its share of the blocks, 16 loads at a time
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t pitch = route_pitch(experts);
    uint32_t quads = 16;
    while (4 * quads < experts) quads *= 2;
    const uint32_t e = tid % quads * 4, part = tid / quads, parts = kRouteThreads / quads;
    if (e < experts) {
        u32x4 sum = {0, 0, 0, 0}, mine = {0, 0, 0, 0};
        for (uint32_t b0 = part; b0 < gridDim.x; b0 += 16 * parts) {
            u32x4 c[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const uint32_t b = b0 + i * parts;
                c[i] = u32x4{0, 0, 0, 0};
                if (i * parts >= gridDim.x) continue;  // (the same in all threads)
                if (b < gridDim.x) c[i] = *reinterpret_cast<const u32x4 *>(hist + (uint64_t)b * pitch + e);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                sum += c[i];
                if (b0 + i * parts < blockIdx.x) mine += c[i];
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (e + j < experts) {
                atomicAdd(&sh.total[e + j], sum[j]);
                atomicAdd(&sh.before[e + j], mine[j]);
            }
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
#define BSR_ROUTE(V, L)                                                                                          \
    hipLaunchKernelGGL((route_select_kernel<TYPE, V, L>), dim3(grid), dim3(kRouteThreads), 0, s, logits, ld, ids,    \
                       weights, offsets, row_token, pos, tokens, experts, top_k, sigmoid, renorm, scale, hist,    \
                       plan.per_block)
    if (experts <= 64)
        BSR_ROUTE(4, 16);
    else if (experts <= 128)
        BSR_ROUTE(8, 16);
    else if (experts <= 256)
        BSR_ROUTE(8, 32);
    else if (experts <= 512)
        BSR_ROUTE(8, 64);
    else
        BSR_ROUTE(16, 64);
#undef BSR_ROUTE
}

// ---------------------------------------------------------------- combine

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
    if (combine_columns(y, residual, out, n) == 8) {
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
