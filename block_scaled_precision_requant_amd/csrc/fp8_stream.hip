// fp8_stream.hip -- the FP8 products for one to a few rows (dense, or per expert), where
// reading the weight once is all the time there is.
//
// out[i,j] = sum_b fl32(a_s[i,b] * w_s[j/128,b]) * P[i,j,b], P the dot product of
// block b.  A workgroup owns 16 rows by 16 columns (with the SiLU product 16 of the gate
// and 16 of the up half) and its waves split K.  A scale block is one K step of
// v_mfma_f32_16x16x128_f8f6f4 (what it adds in fewer than 32 bits: fp8_tile.h), whose
// operand is 32 consecutive codes of a row per lane: the weight rows, and the activations
// beside them, stream from memory straight into the registers that the matrix core reads
// -- no LDS, no swap, no barrier before the end -- two chunks of 128 in flight while the
// two before them are computed.  The weight is the matrix core's row operand, so a lane
// holds four columns of one activation row, whose scale is one value per lane, and the
// weight's is one per wave.  At the end the waves' sums are added in wave order through
// LDS.
//
// In this layout a load touches 16 rows and moves 16 bytes a clock and CU, 9.7 TB/s over
// the chip: enough for the weight alone, which is why rows past kFp8Few run in the tiles
// of fp8_tile.h.  MI355X: one row, n 28672, k 4096 / 8192 (117 / 235 MB) 23.2 / 45.5 us,
// 5.0 TB/s, as a device copy of 1 GiB reaches; n 4096, k 14336 (59 MB, which the 256 MB
// cache holds between calls) 11.2 us; 256 rows through the gate and up projections of 64
// uneven experts, n 4096, k 2048, 82 us.
#include "fp8_internal.h"

namespace bsr {
namespace {

constexpr int kPass = 2;  // chunks in flight

template <int CT>
struct Fp8Pass {
    v8i w[kPass][CT], a[kPass];
    float s[kPass];
};

__device__ __forceinline__ v8i load32(__amdgpu_buffer_rsrc_t r, uint32_t lane_offset, uint32_t offset) {
    return __builtin_shufflevector(load16(r, lane_offset, offset), load16(r, lane_offset + 16, offset), 0, 1, 2, 3, 4,
                                   5, 6, 7);
}

template <bool SILU>
__global__ __launch_bounds__(kFp8MaxWaves * 64, 2) void fp8_stream_kernel(
    const uint8_t *__restrict__ a, const uint8_t *__restrict__ w, const float *__restrict__ a_s,
    const float *__restrict__ w_s, uint16_t *__restrict__ out, GroupedRows g, uint32_t n, uint32_t k,
    uint32_t col_tiles, uint32_t chunks_per_wave, bool wide) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    constexpr int CT = SILU ? 2 : 1;  // weight tiles: a gate and an up tile
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nwaves = blockDim.x >> 6;
    RowTile t = RowTiles(g, 16, lane).find(blockIdx.x / col_tiles);
    t.expert = __builtin_amdgcn_readfirstlane(t.expert);
    t.row0 = __builtin_amdgcn_readfirstlane(t.row0);
    t.rows = __builtin_amdgcn_readfirstlane(t.rows);
    if (t.rows == 0) return;
    const uint32_t c = lane & 15, q = lane >> 4, nb = k / kFp8Block;
    const uint32_t col0 = blockIdx.x % col_tiles * 16, half = n / 2, cols = SILU ? half : n;
    const uint32_t live = min(cols - col0, 16u);
    const uint32_t first = wave * chunks_per_wave, end = min(nb, first + chunks_per_wave);

    // descriptors and scalar offsets, the same in all lanes, and a 32-bit offset per
    // lane; a row outside the buffer reads as 0
    const uint64_t wrow = (uint64_t)t.expert * n + col0;
    const auto rw = __builtin_amdgcn_make_buffer_rsrc((void *)(w + wrow * k), (short)0, (int)(live * k), kRsrcWord3);
    const auto ru = __builtin_amdgcn_make_buffer_rsrc((void *)(w + (wrow + (SILU ? half : 0)) * k), (short)0,
                                                      (int)(live * k), kRsrcWord3);
    const uint32_t wo = c * k + 32 * q;
    const uint32_t blocks = (n + kFp8Block - 1) / kFp8Block;
    const float *ws = w_s + ((uint64_t)t.expert * blocks + col0 / kFp8Block) * nb;
    const float *wsu = w_s + ((uint64_t)t.expert * blocks + ((SILU ? half : 0) + col0) / kFp8Block) * nb;
    const uint32_t arows = g.index != nullptr ? g.src_rows : t.rows;
    const uint64_t a0 = g.index != nullptr ? 0 : t.row0;
    const auto ra = __builtin_amdgcn_make_buffer_rsrc((void *)(a + a0 * k), (short)0, (int)(arows * k), kRsrcWord3);
    const auto rs = __builtin_amdgcn_make_buffer_rsrc((void *)(a_s + a0 * nb), (short)0, (int)(arows * nb * 4), kRsrcWord3);
    uint32_t src = ~0u;
    if (c < t.rows) src = g.index != nullptr ? (uint32_t)g.index[t.row0 + c] : c;
    const uint32_t ao = src < arows ? src * k + 32 * q : kPastEnd;
    const uint32_t so = src < arows ? src * nb * 4 : kPastEnd;

    using Pass = Fp8Pass<CT>;
    // chunks from `chunk` on; past the wave's last one that is read again, and counts 0
    auto load = [&](Pass &b, uint32_t chunk) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
            const uint32_t at = min(chunk + i, end - 1);
#pragma unroll
            for (int j = 0; j < CT; ++j) b.w[i][j] = load32(j == 0 ? rw : ru, wo, at * kFp8Block);
            b.a[i] = load32(ra, ao, at * kFp8Block);
            b.s[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, so, at * 4, 0));
        }
    };
    v4f acc[CT];
#pragma unroll
    for (int j = 0; j < CT; ++j) acc[j] = v4f{0, 0, 0, 0};
    auto compute = [&](const Pass &b, uint32_t chunk) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
            const uint32_t at = min(chunk + i, end - 1);
#pragma unroll
            for (int j = 0; j < CT; ++j) {
                const float s = chunk + i < end ? b.s[i] * (j == 0 ? ws[at] : wsu[at]) : 0.0f;
                const v4f p = fp8_dot16(b.w[i][j], b.a[i]);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[j][r] = fmaf(p[r], s, acc[j][r]);
            }
        }
    };
    // `more`: the next pass's loads go out before this one is computed (a constant at
    // each call: a load that may or may not have been issued would make every later
    // wait the longer one)
    auto pass = [&](Pass &b, Pass &next, uint32_t chunk, bool more) __attribute__((always_inline)) {
        if (more) load(next, chunk + kPass);
        compute(b, chunk);
    };
    Pass b0, b1;
    uint32_t chunk = first;
    const uint32_t last = first + (end - first - 1) / kPass * kPass;
    load(b0, chunk);
    for (;;) {
        if (chunk == last) {
            pass(b0, b1, chunk, false);
            break;
        }
        pass(b0, b1, chunk, true);
        chunk += kPass;
        if (chunk == last) {
            pass(b1, b0, chunk, false);
            break;
        }
        pass(b1, b0, chunk, true);
        chunk += kPass;
    }

    // the waves' sums, added in wave order
    v4f *sums = reinterpret_cast<v4f *>(smem);
#pragma unroll
    for (int j = 0; j < CT; ++j) sums[(wave * CT + j) * 64 + lane] = acc[j];
    __syncthreads();
    if (wave != 0 || c >= t.rows) return;
    v4f v = v4f{0, 0, 0, 0}, up = v;
    for (int x = 0; x < nwaves; ++x) {
        v += sums[x * CT * 64 + lane];
        if constexpr (SILU) up += sums[(x * CT + 1) * 64 + lane];
    }
    if constexpr (SILU)
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = silu_product(v[r], up[r]);
    store4(out, t.row0 + c, col0 + 4 * q, cols, v, wide);
}

}  // namespace

hipError_t launch_fp8_stream(const Fp8Args &p, const Fp8StreamPlan &plan, hipStream_t s) {
    const uint32_t cols = p.silu ? p.n / 2 : p.n;
    const bool wide = cols % 4 == 0 && reinterpret_cast<uintptr_t>(p.out) % 8 == 0;
    auto kernel = p.silu ? fp8_stream_kernel<true> : fp8_stream_kernel<false>;
    hipLaunchKernelGGL(kernel, dim3(plan.row_tiles * plan.col_tiles), dim3(64 * plan.waves), plan.lds, s, p.a, p.w, p.a_s,
                       p.w_s, p.out, p.rows, p.n, p.k, plan.col_tiles, plan.chunks_per_wave, wide);
    return hipGetLastError();
}

}  // namespace bsr
