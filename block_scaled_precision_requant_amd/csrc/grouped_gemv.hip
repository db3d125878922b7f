// grouped_gemv.hip -- the products of grouped.hip for few rows per expert, where
// reading the used experts' weights and scales once is all the time there is.
//
// A workgroup owns 16 columns of one expert and up to 16 (or 4) of its rows;
// its waves split K, so even one row of one expert spreads over the chip, and
// the weight rows stream straight into registers, two 128-byte chunks of each
// in flight while the two before them are computed.  A lane loads block l / 16
// (32 bytes) of weight row l % 16 of a chunk; eight lane swaps turn the chunk's
// 4 x 4 units of 8 bytes, so that one v_mfma_i32_16x16x32_i8 per block gives
// the exact P of 16 activation rows by 16 columns.  Each wave stages the
// activations and their scales of its own pass in LDS; the waves meet at the
// end, where their FP32 sums are added in wave order.
//
// MI355X: one row through each of 8 experts, n 4096, k 2048 (75.6 MB) 15.5-16 us, 4.7-4.9
// TB/s; through 2 experts, n 4096, k 14336 (132 MB) 29 us, 4.5 TB/s; a device copy of 1 GiB
// reaches 5.1 TB/s.
#include "moe_internal.h"

namespace bsr {
namespace {

typedef int v2i __attribute__((ext_vector_type(2)));

struct Pass {
    v4i w[kGgPass][2];
    v4i s[kGgPass];  // scales of the lane's column, one per block
};

template <int ROWS>
__global__ __launch_bounds__(gg_max_waves(ROWS) * 64) void grouped_gemv_kernel(
    const int8_t *__restrict__ a, const int8_t *__restrict__ w, const float *__restrict__ a_s,
    const float *__restrict__ w_s, uint16_t *__restrict__ out, GroupedRows g, uint32_t n, uint32_t k,
    uint32_t col_tiles, uint32_t chunks_per_wave) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    constexpr uint32_t PC = kGgPass, kPitch = gg_pitch(), kBlocks = PC * 4;
    constexpr int kLoads = ROWS * (int)PC / 8;        // 16-byte activation loads per lane and pass ...
    constexpr int kRowLoads = PC * kGgChunk / 16;     // ... of which a row takes this many lanes
    constexpr int kScaleLoads = (ROWS * (int)kBlocks + 63) / 64;
    static_assert(kLoads >= 1 && kRowLoads * ROWS == 64 * kLoads, "whole loads");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nwaves = blockDim.x >> 6;
    RowTile t = RowTiles(g, ROWS, lane).find(blockIdx.x / col_tiles);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.rows == 0) return;
    const uint32_t c = lane & 15, q = lane >> 4, nb = k / 32;
    const uint32_t col0 = blockIdx.x % col_tiles * kGgCols, live = min(n - col0, kGgCols);
    const uint32_t chunks = (k + kGgChunk - 1) / kGgChunk;
    const uint32_t first = wave * chunks_per_wave, end = min(chunks, first + chunks_per_wave);

    // descriptors and scalar offsets, the same in all lanes; a 32-bit offset per
    // lane.  What lies past a buffer reads as 0.
    const uint64_t row = (uint64_t)t.expert * n + col0;
    const auto rw = __builtin_amdgcn_make_buffer_rsrc((void *)(w + row * k), (short)0, (int)(live * k), kRsrcWord3);
    const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)(w_s + row * nb), (short)0, (int)(live * nb * 4), kRsrcWord3);
    const uint32_t wo = c * k + 32 * q, so = c * nb * 4;
    // activations: gathered rows by offset into the whole operand, else from the tile's first row
    const uint32_t arows = g.index != nullptr ? g.src_rows : t.rows;
    const uint64_t a0 = g.index != nullptr ? 0 : t.row0;
    const auto ra = __builtin_amdgcn_make_buffer_rsrc((void *)(a + a0 * k), (short)0, (int)(arows * k), kRsrcWord3);
    const auto rq = __builtin_amdgcn_make_buffer_rsrc((void *)(a_s + a0 * nb), (short)0, (int)(arows * nb * 4), kRsrcWord3);
    auto source = [&](uint32_t r) -> uint32_t {  // operand row of tile row r, ~0 for a row of zeros
        if (r >= t.rows) return ~0u;
        if (g.index == nullptr) return r;
        const uint32_t i = (uint32_t)g.index[t.row0 + r];
        return i < g.src_rows ? i : ~0u;
    };
    uint32_t ao[kLoads], qo[kScaleLoads];
    const uint32_t ak = lane % kRowLoads * 16;  // byte within the pass
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const uint32_t src = source((64 * i + lane) / kRowLoads);
        ao[i] = src == ~0u ? kPastEnd : src * k + ak;
    }
#pragma unroll
    for (int i = 0; i < kScaleLoads; ++i) {
        const uint32_t src = source((64 * i + lane) / kBlocks);
        qo[i] = src == ~0u ? kPastEnd : (src * nb + lane % kBlocks) * 4;
    }

    uint8_t *xs = smem + wave * gg_wave_bytes(ROWS);
    float *qs = reinterpret_cast<float *>(xs + ROWS * kPitch);  // [block][row]
    v4i xv[kLoads];
    float qv[kScaleLoads];
    // (in a pass cut short scalar offsets stay inside a row, and scales come one
    // by one, so that a buffer's end bounds every load)
    auto load = [&](Pass &b, uint32_t chunk, bool part) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (int)PC; ++i) {
            const uint32_t at = min(chunk + i, part ? chunks - 1 : ~0u);
            if (!part) {
                b.s[i] = load16(rs, so, at * 16);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    b.s[i][j] = (int)__builtin_amdgcn_raw_buffer_load_b32(rs, so + 4 * j, at * 16, 0);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) b.w[i][h] = load16(rw, wo + 16 * h, at * kGgChunk);
        }
    };
    // past K in a pass cut short the activations and their scales are 0
    auto load_x = [&](uint32_t chunk, bool part) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            xv[i] = load16(ra, part && chunk * kGgChunk + ak >= k ? kPastEnd : ao[i], chunk * kGgChunk);
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i)
            qv[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
                rq, part && chunk * 4 + lane % kBlocks >= nb ? kPastEnd : qo[i], chunk * 16, 0));
    };
    auto store_x = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            *reinterpret_cast<v4i *>(xs + (64 * i + lane) / kRowLoads * kPitch + ak) = xv[i];
#pragma unroll
        for (int i = 0; i < kScaleLoads; ++i)
            if (ROWS * (int)kBlocks >= 64 || lane < ROWS * (int)kBlocks)
                qs[lane % kBlocks * ROWS + (64 * i + lane) / kBlocks] = qv[i];
    };
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const uint8_t *xa = xs + c % ROWS * kPitch + 8 * q;
    const float *qa = qs + 4 * q % ROWS;
    auto compute = [&](const Pass &b, uint32_t chunks_live) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < (int)PC; ++i) {
            if ((uint32_t)i >= chunks_live) break;
            asm volatile("" ::: "memory");  // a chunk's reads stay with it: bounds live registers
            const v4i w0 = b.w[i][0], w1 = b.w[i][1];
            const v4i even = swap_quarters(v4i{w0.x, w0.z, w1.x, w1.z}), odd = swap_quarters(v4i{w0.y, w0.w, w1.y, w1.w});
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long av = *reinterpret_cast<const long *>(xa + i * kGgChunk + 32 * j);
                const v4f as = *reinterpret_cast<const v4f *>(qa + (4 * i + j) * ROWS);
                const v4i p = __builtin_amdgcn_mfma_i32_16x16x32_i8(av, __builtin_bit_cast(long, v2i{even[j], odd[j]}),
                                                                    v4i{0, 0, 0, 0}, 0, 0, 0);
                const float ws = __int_as_float(b.s[i][j]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[r] = fmaf((float)p[r], as[r] * ws, acc[r]);
            }
        }
    };
    // One whole pass; `more`: the next one is whole too, and its loads go out
    // before this one is computed (a constant at each call: a load that may or
    // may not have been issued would make every later wait the longer one).
    auto pass = [&](Pass &b, Pass &next, uint32_t chunk, bool more) __attribute__((always_inline)) {
        store_x();
        if (more) {
            load_x(chunk + PC, false);
            load(next, chunk + PC, false);
        }
        compute(b, PC);
    };
    const uint32_t whole = min(end, k / kGgChunk);
    const uint32_t passes = first < whole ? (whole - first) / PC : 0;
    Pass b0, b1;
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
        store_x();
        compute(b0, end - chunk);
    }

    // the waves' sums, added in wave order
    __syncthreads();
    v4f *sums = reinterpret_cast<v4f *>(smem);
    sums[wave * 64 + lane] = v4f{acc[0], acc[1], acc[2], acc[3]};
    __syncthreads();
    if (wave != 0) return;
    for (int v = 1; v < nwaves; ++v)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] += sums[v * 64 + lane][r];
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (4 * q + r < t.rows && c < live) out[(uint64_t)(t.row0 + 4 * q + r) * n + col0 + c] = f32_to_bf16_rne(acc[r]);
}

}  // namespace

hipError_t launch_grouped_gemv(const int8_t *a, const int8_t *w, const float *a_s, const float *w_s, uint16_t *out,
                               const GroupedRows &g, uint32_t n, uint32_t k, const GroupedGemvPlan &plan,
                               hipStream_t s) {
    auto kernel = plan.rows == kGgFew ? grouped_gemv_kernel<kGgFew> : grouped_gemv_kernel<kGgRows>;
    hipLaunchKernelGGL(kernel, dim3(plan.row_tiles * plan.col_tiles), dim3(64 * plan.waves), plan.lds, s, a, w, a_s,
                       w_s, out, g, n, k, plan.col_tiles, plan.chunks_per_wave);
    return hipGetLastError();
}

}  // namespace bsr
