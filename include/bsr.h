/*
 * bsr.h -- C ABI of the MI355X (gfx950) block-scaled int8 projection library.
 *
 * The projection Y[M,N] = A[M,K] * W[N,K]^T runs in three steps, each one
 * entry point below:
 *   1. requant_w_nvfp4_int8  -- one-time: NVFP4 weight -> int8 + F32 per 32;
 *   2. requant_a_int8        -- per call: BF16 activations -> int8 + F32 per 32;
 *   3. int8_gemm_blockscaled -- int8 x int8 with an exact int32 dot product per
 *      32-wide K block, each block rescaled in FP32 by a_scale * w_scale,
 *      accumulated in FP32 and written as BF16 (a weight-streaming GEMV for
 *      M <= 16, and up to M = 48 on narrow grids; an MFMA GEMM otherwise).
 * The operations are those of page "metrale_model_layers/layers/ops/
 * gemm_dense_int8.rs": the doc comments of `requant_w_nvfp4_int8` and
 * `int8_gemm_faith2_prefill` (the latter's two launches are entry points 2
 * and 3 here).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensors are dense row-major DEVICE buffers owned by the caller; the
 *   library allocates nothing, keeps no pointer after it returns and never
 *   synchronises.  Host pointers are not accepted (undefined behaviour).
 * - Work is enqueued on `stream` (a hipStream_t passed as void*, NULL = the
 *   default stream).  Calls on one stream run in order, so the output of
 *   requant_a_int8 may be passed straight to int8_gemm_blockscaled.
 * - Sizes are uint32_t; index arithmetic inside is 64-bit.
 * - Validation happens before any launch: on an error nothing is launched and
 *   no output byte is written.  There is no fallback to another path.
 * - m == 0 or n == 0 is a valid empty problem: BSR_OK, nothing launched.
 * - k must be a positive multiple of 32 (every K/2, K/16, K/32 is whole).
 * - Inputs outside the method's contract (NaN/Inf activations, NaN E4M3
 *   scale codes, a non-finite dequantized weight) give unspecified output.
 * - Outputs must not alias inputs (undefined behaviour, not checked).
 * - The calling thread's current HIP device must be a gfx950 GPU; the device
 *   check is cached per device, so the library is safe to call from several
 *   host threads.
 *
 * Number formats: E2M1 per the OCP Microscaling Formats v1.0 spec, element
 * 2j of a packed byte row in the LOW nibble of byte j; E4M3 per the OCP 8-bit
 * floating point spec (no infinities, S.1111.111 NaN); BF16 = upper half of
 * an IEEE binary32.
 *
 * Quantizer (steps 1 and 2), per 32-element block of a row:
 *   amax = max |v|;  s = fl32(amax / 127) (IEEE divide), stored as the scale;
 *   s == 0 (zero block or underflow): scale +0.0f and q = 0;
 *   else q = clamp(round_half_even(fl32(v / s)), -127, 127).
 * Results are bit-identical to that definition (subnormals included).
 */
#ifndef BSR_H
#define BSR_H

#include <stdint.h>

/* The library is built with hidden visibility: exactly the functions declared
 * here are exported from libbsr.so. */
#if defined(__GNUC__) || defined(__clang__)
#define BSR_API __attribute__((visibility("default")))
#else
#define BSR_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
enum bsr_status {
    BSR_OK = 0,
    BSR_EINVAL = 1,  /* k == 0, k % 32 != 0, unsupported size, or bad `path` */
    BSR_ENULL = 2,   /* a required pointer is NULL (m, n > 0)                */
    BSR_EALIGN = 3,  /* a pointer is not aligned as stated per argument      */
    BSR_EDEVICE = 4, /* no current HIP device, or it is not gfx950           */
    BSR_ELAUNCH = 5  /* the kernel launch reported an error                  */
};

/*
 * Step 1, one-time weight requant (page ".../gemm_dense_int8.rs", doc of
 * `requant_w_nvfp4_int8`).
 *   w_packed [n, k/2]  u8  two E2M1 codes per byte, low nibble first; 16-byte aligned
 *   w_e4m3   [n, k/16] u8  E4M3 scale of elements 16c..16c+15;       2-byte aligned
 *   scale2             f32 per-tensor scale, by value; must be finite
 *   w_i8     [n, k]    i8  output codes in [-127, 127];              16-byte aligned
 *   w_scale  [n, k/32] f32 output scale of each 32-block;             4-byte aligned
 * Dequantized value: v = fl32(fl32(e2m1 * e4m3) * scale2) (the first product
 * is exact), then the quantizer above.
 * Errors: BSR_EINVAL (k, or scale2 not finite), BSR_ENULL, BSR_EALIGN,
 * BSR_EDEVICE, BSR_ELAUNCH.
 */
BSR_API int requant_w_nvfp4_int8(const uint8_t *w_packed, const uint8_t *w_e4m3, float scale2,
                                 int8_t *w_i8, float *w_scale, uint32_t n, uint32_t k, void *stream);

/*
 * Step 2, per-call activation requant (page ".../gemm_dense_int8.rs", doc of
 * `int8_gemm_faith2_prefill`, its first launch).
 *   a_bf16  [m, k]    BF16 as raw u16;  16-byte aligned
 *   a_i8    [m, k]    i8 output;        16-byte aligned (caller-owned scratch)
 *   a_scale [m, k/32] f32 output;        4-byte aligned (caller-owned scratch)
 * Errors: BSR_EINVAL, BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.
 */
BSR_API int requant_a_int8(const uint16_t *a_bf16, int8_t *a_i8, float *a_scale,
                           uint32_t m, uint32_t k, void *stream);

/*
 * Step 3, block-scaled GEMM (page ".../gemm_dense_int8.rs", doc of
 * `int8_gemm_faith2_prefill`, its second launch).
 *   a_i8    [m, k]    i8,  16-byte aligned     w_i8    [n, k]    i8,  16-byte aligned
 *   a_scale [m, k/32] f32,  4-byte aligned     w_scale [n, k/32] f32,  4-byte aligned
 *   out     [m, n]    BF16 as raw u16, 2-byte aligned
 * out[i,j] = bf16_rne( FP32 sum over blocks b of fl32(a_scale[i,b] * w_scale[j,b])
 *            * P[i,j,b] ), P the exact int32 dot product of block b.  The FP32
 * summation order is the kernel's own (not part of the contract); the result
 * is within 4e-3 relative or 1 BF16 ulp of the FP64 value, or within the
 * worst-case FP32 error of a K/32-term sum where that is larger.
 * Scales must be finite: a NaN or Inf in a_scale or w_scale is outside the
 * contract and may make other rows' outputs non-finite too (the kernels read
 * a few scales past a row's last block and zero their products by
 * multiplying by 0).
 * m <= 16 (one 16-row matrix-core tile) runs the weight-streaming GEMV; so
 * does m <= 48 when k is a multiple of 256 and n <= 4096 (16-column
 * workgroups at most one per CU); other shapes run the MFMA GEMM.
 * Limit: for m > 16, k < 2^25 (the GEMM addresses a tile's 128 rows with
 * 32-bit offsets).
 * Errors: BSR_EINVAL (k; m > 16 with k >= 2^25), BSR_ENULL, BSR_EALIGN,
 * BSR_EDEVICE, BSR_ELAUNCH.
 */
BSR_API int int8_gemm_blockscaled(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                                  const float *w_scale, uint16_t *out, uint32_t m, uint32_t n,
                                  uint32_t k, void *stream);

/* Paths of int8_gemm_blockscaled_ex. */
enum bsr_path {
    BSR_PATH_AUTO = 0, /* as int8_gemm_blockscaled                       */
    BSR_PATH_GEMM = 1, /* the MFMA GEMM at any m (k < 2^25)              */
    BSR_PATH_GEMV = 2, /* the GEMV; requires m <= 16, or m <= 64 with k a
                        * multiple of 256, else BSR_EINVAL              */
    BSR_PATH_INVARIANT = 3 /* m <= 16: a GEMV that accumulates every output
                            * over the K blocks in increasing order, as the
                            * GEMM does; m > 16: the GEMM.  A row's output
                            * bits then depend on neither m nor the path
                            * (the invariants stated for `W8a8Weight::segment`
                            * on page "metrale_model_layers/layers/ops/
                            * w8a8_decode/parts.rs" and for `nvfp4_proj_mx`
                            * on page ".../w4a4_proj/fixed.rs"); slower
                            * decode than BSR_PATH_GEMV, whose waves split K */
};

/*
 * int8_gemm_blockscaled with an explicit path, so tests can run both kernels
 * on the same rows (same arguments and errors; BSR_EINVAL for an unknown path).
 */
BSR_API int int8_gemm_blockscaled_ex(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                                     const float *w_scale, uint16_t *out, uint32_t m, uint32_t n,
                                     uint32_t k, void *stream, int path);

/*
 * Workspace bytes int8_gemm_blockscaled_ws needs for an (m, n, k) problem: 0
 * when that problem runs without a K split (then no workspace is used), else
 * at most 8 MiB.  Pure host arithmetic, no device call.
 */
BSR_API uint64_t int8_gemm_blockscaled_ws_bytes(uint32_t m, uint32_t n, uint32_t k);

/*
 * int8_gemm_blockscaled with a caller workspace, for grids too small to fill
 * the GPU: m > 32 rows in fewer 64 x 64 output tiles than compute units with
 * k >= 8192 (e.g. m = 48..192 at n = 4096, k = 14336), where it measured
 * faster than the paths without workspace.  Each tile's K range is cut into
 * slices of whole 128-element
 * stages, one workgroup per (tile, slice), each writing its FP32 tile to the
 * workspace; a second launch adds the slices in slice order and rounds to
 * BF16.  Same step as the GEMM launch of `int8_gemm_faith2_prefill` (page
 * "metrale_model_layers/layers/ops/gemm_dense_int8.rs"); the FP32 sum per
 * output is (sum over the slices, in order, of each slice's chain over its
 * blocks), within the same tolerance as int8_gemm_blockscaled.  Problems
 * with no split (int8_gemm_blockscaled_ws_bytes == 0) run exactly as
 * int8_gemm_blockscaled and do not touch the workspace.
 *   arguments 1-8 as int8_gemm_blockscaled
 *   workspace        device buffer of workspace_bytes, 16-byte aligned; its
 *                    contents on entry do not matter, on return they are
 *                    scratch; it must not alias any other argument, and two
 *                    calls that may overlap in time must not share it
 * Errors: as int8_gemm_blockscaled; when a split runs, BSR_ENULL (workspace
 * NULL), BSR_EALIGN (workspace), BSR_EINVAL (workspace_bytes below
 * int8_gemm_blockscaled_ws_bytes(m, n, k)).
 */
BSR_API int int8_gemm_blockscaled_ws(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                                     const float *w_scale, uint16_t *out, uint32_t m, uint32_t n, uint32_t k,
                                     void *workspace, uint64_t workspace_bytes, void *stream);

/*
 * int8_gemm_blockscaled_ws for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the K-split workspace is the library's own static device array
 * of 8 MiB per GPU (the most any split plan asks for), held until the process
 * ends; the call allocates nothing.  Same arguments as int8_gemm_blockscaled
 * and the same results as int8_gemm_blockscaled_ws, bit for bit.
 * Every call on one GPU shares that GPU's array: calls that may overlap in
 * time on one GPU (different streams, or several host threads) race and give
 * undefined results; calls ordered on one stream do not.  Nothing in the
 * array must start at zero (each call overwrites what it reads).
 * Errors: as int8_gemm_blockscaled; BSR_EINVAL if a split would need more
 * than the 8 MiB array (no problem size does); BSR_EDEVICE if the array's
 * device address cannot be obtained.
 */
BSR_API int int8_gemm_blockscaled_noalloc(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                                          const float *w_scale, uint16_t *out, uint32_t m, uint32_t n,
                                          uint32_t k, void *stream);

/*
 * Fused SiLU·mul -> int8 per-32 requant: the quantized input of the down
 * projection, straight from the gate and up halves of a gate+up output (the
 * SiLU-product quantizer `W8a8Kernels::quant_silu` of page
 * "metrale_model_layers/layers/ops/w8a8_decode/parts.rs" and the re-quantized
 * SiLU product of page ".../fp8_moe_grouped_tc_w8a8.rs", here with the int8
 * per-32 quantizer of step 2).
 *   gate, up [m, ld] BF16 as raw u16, 16-byte aligned; columns 0..k-1 of each
 *            row are used (ld >= k, ld a multiple of 8).  Both halves of one
 *            [m, 2I] buffer qualify: gate = buf, up = buf + I, ld = 2I.
 *   a_i8     [m, k]    i8 output, dense, 16-byte aligned
 *   a_scale  [m, k/32] f32 output, dense, 4-byte aligned
 * Per element: e = exp(-g) rounded once to binary32 (evaluated in binary64),
 * h = bf16_rne(fl32(fl32(g / fl32(1 + e)) * u)); then the quantizer above on
 * the 32-blocks of h, so the result equals requant_a_int8 applied to the BF16
 * SiLU product.  (Where exp(-g) overflows binary32, g < -88.72, silu is -0.)
 * Errors: BSR_EINVAL (k, ld < k, ld not a multiple of 8), BSR_ENULL,
 * BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.
 */
BSR_API int silu_mul_requant_int8(const uint16_t *gate, const uint16_t *up, uint32_t ld, int8_t *a_i8,
                                  float *a_scale, uint32_t m, uint32_t k, void *stream);

/*
 * W4A16 decode GEMV straight from the NVFP4 weight, no int8 requant (the
 * decode launcher of page "metrale_model_layers/layers/ops/gemv_sw.rs":
 * BF16 input, packed weight, E4M3 weight scale, F32 scale_2, BF16 output).
 *   x_bf16   [m, k]    BF16 as raw u16, 16-byte aligned, 1 <= m <= 16
 *   w_packed [n, k/2]  u8 (E2M1 pairs, low nibble first), 16-byte aligned
 *   w_e4m3   [n, k/16] u8, 16-byte aligned when k % 256 == 0, else 2-byte
 *   out      [m, n]    BF16 as raw u16, 2-byte aligned
 * out[i,j] = bf16_rne( fl32( S * scale2 ) ), S an FP32 evaluation of the sum
 * over k of x[i,k] * e2m1[j,k] * s16[j,k/16] in the kernel's own order (for
 * k % 256 == 0 the exact products x * e2m1 are summed per 16-element scale
 * block and each block sum is multiplied by its s16; otherwise the exact
 * products x * (e2m1 * s16) are summed): within 4e-3 relative or 1 BF16 ulp
 * of the FP64 value, or within the worst-case FP32 error of a (k + 16)-term
 * sum.
 * Errors: BSR_EINVAL (k, m > 16, scale2 not finite), BSR_ENULL, BSR_EALIGN,
 * BSR_EDEVICE, BSR_ELAUNCH.
 */
BSR_API int w4a16_gemv(const uint16_t *x_bf16, const uint8_t *w_packed, const uint8_t *w_e4m3, float scale2,
                       uint16_t *out, uint32_t m, uint32_t n, uint32_t k, void *stream);

/* Activation code formats of quantize_act. */
enum bsr_format {
    BSR_FMT_INT8 = 0, /* int8 codes, scale = amax / 127                    */
    BSR_FMT_E4M3 = 1  /* OCP E4M3 codes (bias 7, max 448), amax / 448      */
};

/*
 * Activation quantizer with another scale layout: one F32 scale per group of
 * `group` consecutive elements of a row (32 or 128) or per row (group = 0),
 * int8 or E4M3 codes (the W8A8 activation layouts `W8a8Scale::PerRow` /
 * `W8a8Scale::Block128` and the FP8 activation of page
 * "metrale_model_layers/layers/ops/w8a8_decode/parts.rs"; the per-(row, 128)
 * E4M3 quantizer of page ".../fp8_moe_grouped_tc_w8a8.rs").
 *   a_bf16 [m, k]         BF16 as raw u16, 16-byte aligned, k % 32 == 0
 *                         (k % 128 == 0 for group 128)
 *   q      [m, k]         u8 codes (int8 two's complement or E4M3), 8-byte aligned
 *   scale  [m, k / group] F32 ([m] for group 0), 4-byte aligned
 * Per group: s = fl32(amax / F), F = 127 (int8) or 448 (E4M3); s == 0 gives
 * scale +0 and codes 0; else q = clamp(rne(fl32(v / s)), -127, 127) for int8
 * and the E4M3 code nearest fl32(v / s) (ties to the even code) for E4M3.
 * group 32 with BSR_FMT_INT8 equals requant_a_int8.
 * Errors: BSR_EINVAL (k, group, format), BSR_ENULL, BSR_EALIGN, BSR_EDEVICE,
 * BSR_ELAUNCH.
 */
BSR_API int quantize_act(const uint16_t *a_bf16, uint8_t *q, float *scale, uint32_t m, uint32_t k,
                         uint32_t group, int format, void *stream);

/*
 * int8_gemm_blockscaled_ex with int8 activations whose scales come per group
 * of a_group elements (32 or 128) or per row (a_group = 0), as quantize_act
 * writes them: block b of row r is rescaled by fl32(a_scale[r, (32 b) /
 * a_group] * w_scale[n, b]) (a_scale[r] for a_group 0), so the result equals
 * int8_gemm_blockscaled with each activation scale repeated over its blocks.
 *   a_scale [m, k / a_group] F32 ([m] for a_group 0), 4-byte aligned
 * Other arguments, path and the output tolerance as int8_gemm_blockscaled_ex.
 * Errors: BSR_EINVAL (a_group not 0/32/128, a_group 128 with k % 128 != 0,
 * or as int8_gemm_blockscaled_ex), BSR_ENULL, BSR_EALIGN, BSR_EDEVICE,
 * BSR_ELAUNCH.
 */
BSR_API int int8_gemm_blockscaled_agroup(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                                         uint32_t a_group, const float *w_scale, uint16_t *out, uint32_t m,
                                         uint32_t n, uint32_t k, void *stream, int path);

/* ---- expert layers and integer 4-bit weights ------------------------------
 *
 * One expert layer over tokens [T]: moe_route picks the experts of each token
 * and orders the (token, slot) pairs by expert; the products of the rows of
 * each expert run in int8_grouped_gemm_blockscaled (int8 weights) or
 * w4a16_group_gemv_experts (4-bit weights, decode); moe_combine adds a token's
 * rows with their weights (the grouped W8A8 expert product of page
 * "metrale_model_layers/layers/ops/fp8_moe_grouped_tc_w8a8.rs", with the int8
 * per-32 formats of this library).
 *
 * Rows and experts: the rows [offsets[e], offsets[e + 1]) of a grouped call
 * belong to expert e.  offsets is a DEVICE array of experts + 1 ascending
 * int32 values in [0, rows], so no host synchronisation stands between the
 * router and the products.  It cannot be checked on the host: values outside
 * [0, rows] are clamped, a descending pair is an expert without rows, and
 * where the remaining ranges overlap the output of every row inside them is
 * unspecified (some may not be written at all); no value makes a kernel read or
 * write outside its arguments.  Rows of no range are left as they were.
 */

/* Element types of the arguments that take more than one. */
enum bsr_type { BSR_TYPE_BF16 = 0, BSR_TYPE_F16 = 1, BSR_TYPE_F32 = 2 };

/* Scores of moe_route. */
enum bsr_score {
    BSR_SCORE_SOFTMAX = 0, /* softmax over all experts of the row */
    BSR_SCORE_SIGMOID = 1  /* sigmoid of each logit               */
};

/*
 * Workspace bytes moe_route needs: 0 for few tokens (and for sizes that it
 * refuses), never more than 1024 * experts.  Pure host arithmetic, no device call.
 */
BSR_API uint64_t moe_route_ws_bytes(uint32_t tokens, uint32_t experts, uint32_t top_k);

/*
 * Router: the top_k experts of each token, their weights, and the order of
 * the routed rows by expert.
 *   logits    [tokens, experts] of `type` (enum bsr_type), rows `ld` elements
 *             apart (ld >= experts), aligned to the element
 *   ids       [tokens, top_k] i32  experts by falling logit, ties to the lowest
 *             index; an expert whose logit is -inf or NaN is never taken, and a
 *             slot left over (a padded token's row of -inf) holds -1
 *   weights   [tokens, top_k] f32  scale * score of each id, 0 where it is -1;
 *             renorm != 0: the scores are divided by their sum over the taken ids
 *   offsets   [experts + 1] i32    first row of each expert, then the row count
 *   row_token [tokens * top_k] i32 token of each row; rows of one expert keep
 *             the order of (token, slot); behind the last row left as it was
 *   pos       [tokens, top_k] i32  row of each (token, slot), -1 where id is -1
 *   scale     f32 factor of the weights, finite
 * Scores are evaluated in binary32, a sum of scores as one binary32 tree;
 * +inf logits share the softmax between them.  A softmax's maximum is taken
 * over the row's logits other than NaN.  The result does not depend on the
 * order in which workgroups run.  tokens == 0 writes offsets (all 0) only.
 *   workspace 16-byte aligned device buffer of at least moe_route_ws_bytes, as
 *             that of int8_gemm_blockscaled_ws: scratch, and not shared by
 *             calls that may overlap in time (NULL where 0 bytes are needed)
 * Limits: 1 <= experts <= 1024, 1 <= top_k <= min(16, experts), tokens * top_k
 * < 2^31.
 * Errors: BSR_EINVAL (those limits, ld, type, score, scale, a workspace that is
 * too small), BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.
 */
BSR_API int moe_route(const void *logits, int type, uint32_t ld, int32_t *ids, float *weights, int32_t *offsets,
                      int32_t *row_token, int32_t *pos, uint32_t tokens, uint32_t experts, uint32_t top_k, int score,
                      int renorm, float scale, void *workspace, uint64_t workspace_bytes, void *stream);

/*
 * Block-scaled int8 products grouped by expert, ragged row counts:
 * out[p, j] = bf16_rne( FP32 sum over blocks b of fl32(a_scale[i, b] *
 * w_scale[e, j, b]) * P[i, e, j, b] ) for the rows p of expert e, with i =
 * row_index[p] (i = p where row_index is NULL) and P as for
 * int8_gemm_blockscaled, whose tolerance holds here too.
 *   a_i8    [a_rows, k]         i8,  16-byte aligned
 *   w_i8    [experts, n, k]     i8,  16-byte aligned
 *   a_scale [a_rows, k/32]      f32,  4-byte aligned
 *   w_scale [experts, n, k/32]  f32,  4-byte aligned
 *   offsets [experts + 1]       i32,  4-byte aligned (see above)
 *   row_index [rows] i32 (moe_route's row_token) or NULL; an entry outside
 *           [0, a_rows) stands for a row of zeros.  NULL needs a_rows >= rows,
 *           row_index a_rows >= 1
 *   out     [rows, n]           BF16 as raw u16, 2-byte aligned
 * `rows` is the row capacity (tokens * top_k); offsets says how many are used.
 * Scales must be finite, as for int8_gemm_blockscaled.  The FP32 summation
 * order follows the sizes of the call; equal calls give equal bits.
 * Limits: experts <= 65536, rows < 2^31, k < 2^24, and with row_index a_rows *
 * k < 2^32 (the rows are gathered with 32-bit offsets).
 * Errors: BSR_EINVAL (k, those limits, a_rows too small, a launch of 2^32 threads),
 * BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.  rows == 0, n == 0 or
 * experts == 0 is a valid empty problem.
 */
BSR_API int int8_grouped_gemm_blockscaled(const int8_t *a_i8, const int8_t *w_i8, const float *a_scale,
                                          const float *w_scale, const int32_t *offsets, const int32_t *row_index,
                                          uint16_t *out, uint32_t a_rows, uint32_t rows, uint32_t experts, uint32_t n,
                                          uint32_t k, void *stream);

/*
 * Weighted sum of the experts' rows back into their tokens:
 * out[t] = bf16_rne( residual[t] + sum over slots s of weights[t, s] *
 * y[pos[t, s]] ), in binary32, the residual first and the slots in order; a
 * slot whose pos is outside [0, rows) adds nothing and reads nothing.
 *   y        [rows, n]       BF16 as raw u16, 2-byte aligned
 *   pos      [tokens, top_k] i32, weights [tokens, top_k] f32, 4-byte aligned
 *   residual [tokens, n]     BF16 as raw u16 or NULL, 2-byte aligned
 *   out      [tokens, n]     BF16 as raw u16, 2-byte aligned; may be residual
 * Limits: 1 <= top_k <= 16.
 * Errors: BSR_EINVAL (top_k, a launch of 2^32 threads: one per 8 columns of a
 * token, or per column where n % 8 != 0 or a pointer is not 16-byte aligned, in
 * wholes of 256), BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.  rows == 0 is
 * valid (no slot adds anything).
 */
BSR_API int moe_combine(const uint16_t *y, const int32_t *pos, const float *weights, const uint16_t *residual,
                        uint16_t *out, uint32_t tokens, uint32_t top_k, uint32_t rows, uint32_t n, void *stream);

/*
 * Decode GEMV with integer 4-bit weights and a scale (and zero point) per
 * group of k: out[i, j] = bf16_rne( sum over groups g of scale[j, g] * sum over
 * k in g of x[i, k] * (c[j, k] - z[j, g]) ), c = 0..15.
 *   x        [m, k]       BF16 as raw u16, 16-byte aligned
 *   w_packed [n, k/2]     u8, two codes per byte, element 2j in the LOW nibble
 *                         of byte j; 16-byte aligned
 *   scale    [n, k/group] of scale_type (enum bsr_type), aligned to the element
 *   zero     [n, k/group] u8 zero points 0..255, or NULL: every z is 8
 *   group    32, 64 or 128 (dividing k), or 0: one scale per row of the weight
 *   out      [m, n]       BF16 as raw u16, 2-byte aligned
 * Evaluated in binary32: per group (group 0: per 128 elements) the codes enter
 * as the exact values 16 + c and (16 + z) * sum(x) is taken off, then the scale
 * is applied once, so the error of a sum is bounded with the terms |x| * scale *
 * (32 + c + z).
 * No group's sum overflows for finite x.  A NaN or Inf in x leaves its own row
 * of out unspecified, one in scale its own column (of its expert), no other.
 * Meant for m <= 16; every further 16 rows read the weight once more.
 * Limits: k < 2^24, m * k < 2^31 (the activations are read with 32-bit offsets).
 * Errors: BSR_EINVAL (k, group, scale_type, those limits, a launch of 2^32
 * threads), BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.
 */
BSR_API int w4a16_group_gemv(const uint16_t *x, const uint8_t *w_packed, const void *scale, int scale_type,
                             const uint8_t *zero, uint32_t group, uint16_t *out, uint32_t m, uint32_t n, uint32_t k,
                             void *stream);

/*
 * w4a16_group_gemv by expert: row p of expert e takes the weight of e.
 *   x        [x_rows, k]           w_packed [experts, n, k/2]
 *   scale    [experts, n, k/group] zero     [experts, n, k/group] or NULL
 *   offsets, row_index as int8_grouped_gemm_blockscaled
 *   silu_mul 0: out [rows, n].  1: columns 0..n/2-1 of the weight are the gate
 *            and n/2..n-1 the up projection, out [rows, n/2] =
 *            bf16_rne( fl32(gate / fl32(1 + exp(-gate))) * up ), gate and up in
 *            binary32; n must be even
 * Limits: experts <= 65536, rows < 2^31, k < 2^24, x_rows * k < 2^31.
 * Errors: as w4a16_group_gemv; BSR_EINVAL too for x_rows too small (as a_rows
 * there), silu_mul other than 0 or 1, an odd n with it, and those limits.
 */
BSR_API int w4a16_group_gemv_experts(const uint16_t *x, const uint8_t *w_packed, const void *scale, int scale_type,
                                     const uint8_t *zero, uint32_t group, const int32_t *offsets,
                                     const int32_t *row_index, int silu_mul, uint16_t *out, uint32_t x_rows,
                                     uint32_t rows, uint32_t experts, uint32_t n, uint32_t k, void *stream);

/* ---- FP8 products and rows of sorted tokens ---------------------------------
 *
 * E4M3 codes with F32 scales per 128: activations per (row, 128 elements), as
 * quantize_act writes them (group 128, BSR_FMT_E4M3: the FP8 activation of page
 * "metrale_model_layers/layers/ops/fp8_moe_grouped_tc_w8a8.rs"), weights per block
 * of 128 rows x 128 elements, as quantize_w_fp8 writes them.  Since the blocks are
 * square, the transposed codes with the transposed scales are a weight of the same
 * form: the data gradient of a product is the same product on them.
 */

/*
 * Weight quantizer: BF16 -> E4M3 codes and one scale per block of 128 x 128.
 *   w_bf16    [experts, n, k]               BF16 as raw u16, 16-byte aligned
 *   w_q       [experts, n, k]               u8 E4M3 codes, 16-byte aligned
 *   w_scale   [experts, ceil(n/128), k/128] f32, 4-byte aligned
 *   w_qt      [experts, k, n]               u8, the codes transposed, 16-byte
 *             aligned, or NULL; then n % 128 == 0
 *   w_scale_t [experts, k/128, n/128]       f32, w_scale transposed, 4-byte
 *             aligned; NULL if and only if w_qt is
 * Per block (the last block of rows may be shorter): s = fl32(amax / 448); s == 0
 * gives scale +0 and codes 0, else the E4M3 code nearest fl32(v / s), ties to the
 * even code, at most 448 in magnitude.  A NaN or Inf makes the scale of its own block
 * NaN or Inf, and the block's codes unspecified.
 * Errors: BSR_EINVAL (k == 0, k % 128 != 0, n % 128 != 0 with w_qt, a launch of 2^32
 * threads: 256 per block), BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.
 * experts == 0 or n == 0 is a valid empty problem.
 */
BSR_API int quantize_w_fp8(const uint16_t *w_bf16, uint8_t *w_q, float *w_scale, uint8_t *w_qt, float *w_scale_t,
                           uint32_t experts, uint32_t n, uint32_t k, void *stream);

/*
 * FP8 product: out[i, j] = bf16_rne( FP32 sum over blocks b of 128 elements of
 * fl32(a_scale[i, b] * w_scale[j / 128, b]) * P[i, j, b] ), P the dot product of
 * block b by the FP8 matrix core.
 *   a_q     [m, k]               u8 E4M3 codes, 16-byte aligned
 *   w_q     [n, k]               u8 E4M3 codes, 16-byte aligned
 *   a_scale [m, k/128]           f32, 4-byte aligned
 *   w_scale [ceil(n/128), k/128] f32, 4-byte aligned
 *   out     [m, n]               BF16 as raw u16, 2-byte aligned
 * The matrix core adds the products of 8 consecutive codes in fixed point, each cut
 * below 2^-13 of the largest one's power of two (a code stands for its value to 2^-4,
 * so what is cut is below 1/64 of what the largest code leaves open), and the groups of
 * 8 in binary32.  The result is within 4e-3 relative or 1 BF16 ulp of the FP64 value,
 * or where that is larger within 7 * 2^-13 of the sum over the groups of their largest
 * scaled product, plus the worst-case FP32 error of the sum.  The order of the sum
 * follows the sizes of the call; equal calls give equal bits.  A NaN code, and a
 * scale of NaN or Inf, makes only its own row (a_q, a_scale), column (w_q) or 128
 * columns (w_scale) of out other than finite.
 * Limits: k < 2^23, m and n < 2^31.
 * Errors: BSR_EINVAL (k == 0, k % 128 != 0, those limits, a launch of 2^32 threads),
 * BSR_ENULL, BSR_EALIGN, BSR_EDEVICE, BSR_ELAUNCH.  m == 0 or n == 0 is a valid empty
 * problem.
 */
BSR_API int fp8_gemm_blockscaled(const uint8_t *a_q, const uint8_t *w_q, const float *a_scale, const float *w_scale,
                                 uint16_t *out, uint32_t m, uint32_t n, uint32_t k, void *stream);

/*
 * fp8_gemm_blockscaled grouped by expert, ragged row counts: row p of expert e is
 * operand row row_index[p] (p where row_index is NULL) times the weight of e.
 *   a_q     [a_rows, k]                   a_scale [a_rows, k/128]
 *   w_q     [experts, n, k]               w_scale [experts, ceil(n/128), k/128]
 *   offsets, row_index as int8_grouped_gemm_blockscaled
 *   silu_mul 0: out [rows, n].  1: columns 0..n/2-1 of the weight are the gate and
 *           n/2..n-1 the up projection, out [rows, n/2] = bf16_rne( fl32(gate /
 *           fl32(1 + exp(-gate))) * up ), gate and up in binary32, the value before it is
 *           rounded to BF16 within (1.25 |gate| + 8) 2^-24 of it, or where the quotient is
 *           subnormal within a step of it, 2^-149 |up|; n % 256 == 0
 * Limits: experts <= 65536, rows and n < 2^31, k < 2^23, and with row_index a_rows *
 * k < 2^32 (the rows are gathered with 32-bit offsets).
 * Errors: as fp8_gemm_blockscaled; BSR_EINVAL too for a_rows too small (NULL
 * row_index needs a_rows >= rows, row_index a_rows >= 1), silu_mul other than 0 or 1,
 * n % 256 != 0 with it, and those limits.  rows == 0, n == 0 or experts == 0 is a
 * valid empty problem.
 */
BSR_API int fp8_grouped_gemm_blockscaled(const uint8_t *a_q, const uint8_t *w_q, const float *a_scale,
                                         const float *w_scale, const int32_t *offsets, const int32_t *row_index,
                                         int silu_mul, uint16_t *out, uint32_t a_rows, uint32_t rows, uint32_t experts,
                                         uint32_t n, uint32_t k, void *stream);

/*
 * Rows of tokens copied into the experts' order: out[pos[t, s]] = x[t] for every
 * slot s, for products that take no row_index.  A slot whose pos is outside [0,
 * rows) is skipped; rows of out that no slot names are left as they were.  Where two
 * slots of different tokens name one row (moe_route's pos has no such pair) each
 * element of it is one of theirs.
 *   x   [tokens, n]     BF16 as raw u16, 2-byte aligned
 *   pos [tokens, top_k] i32, 4-byte aligned
 *   out [rows, n]       BF16 as raw u16, 2-byte aligned
 * Limits: 1 <= top_k <= 16, n < 2^31.
 * Errors: BSR_EINVAL (those limits, a launch of 2^32 threads: 256 per 2048 columns of
 * a token, or per slot if those are more), BSR_ENULL, BSR_EALIGN, BSR_EDEVICE,
 * BSR_ELAUNCH.  tokens == 0, n == 0 or rows == 0 is a valid empty problem.
 */
BSR_API int moe_dispatch(const uint16_t *x, const int32_t *pos, uint16_t *out, uint32_t tokens, uint32_t top_k,
                         uint32_t rows, uint32_t n, void *stream);

/*
 * Gradient of moe_dispatch: d_x[t] = bf16_rne( sum over slots s of d_rows[pos[t, s]]
 * ), in binary32, the slots in order; a slot whose pos is outside [0, rows) adds
 * nothing and reads nothing (a token without slots gets 0).
 *   d_rows [rows, n], d_x [tokens, n]  BF16 as raw u16, 2-byte aligned
 * Other arguments, limits and errors as moe_dispatch; rows == 0 gives zeros.
 */
BSR_API int moe_dispatch_grad(const uint16_t *d_rows, const int32_t *pos, uint16_t *d_x, uint32_t tokens,
                              uint32_t top_k, uint32_t rows, uint32_t n, void *stream);

/*
 * Gradient of moe_combine for d_out = dL/d out (that of its residual is d_out):
 * with p = pos[t, s],
 *   d_y[p] = bf16_rne( weights[t, s] * d_out[t] ),
 *   d_weights[t, s] = sum over j of d_out[t, j] * y[p, j], in binary32.
 * A slot whose p is outside [0, rows) has d_weights 0 and touches no row; rows of d_y
 * that no slot names are left as they were.  Where several slots name one row
 * (moe_route's pos has no such pair) each element of it is one of theirs, not the
 * sum, and with d_y = y their d_weights are unspecified.  The order of a sum follows
 * n; equal calls give equal bits.
 *   d_out   [tokens, n]     BF16 as raw u16, 2-byte aligned
 *   y, d_y  [rows, n]       BF16 as raw u16, 2-byte aligned; d_y may be y
 *   pos     [tokens, top_k] i32, weights, d_weights [tokens, top_k] f32, 4-byte aligned
 * Limits and errors as moe_dispatch.  n == 0 and rows == 0 give d_weights of 0.
 */
BSR_API int moe_combine_grad(const uint16_t *d_out, const uint16_t *y, const int32_t *pos, const float *weights,
                             uint16_t *d_y, float *d_weights, uint32_t tokens, uint32_t top_k, uint32_t rows,
                             uint32_t n, void *stream);

/* Human-readable name of a status code (static storage, never NULL). */
BSR_API const char *bsr_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* BSR_H */
