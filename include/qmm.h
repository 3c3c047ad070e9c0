/*
 * qmm.h -- fused dequantize-and-multiply of block-quantized weights on MI355X (gfx950).
 *
 * y = x . W^T, where W (M rows x K) is stored as packed quantized blocks that the
 * kernels decode themselves, x holds N activation tokens of K values, and y is
 * N x M fp32.  This is the operation all three source pages optimise:
 *   - candle pull request "Metal: 64-token tile for the quantized matrix-matrix
 *     kernel" (sections "What changes" and "Why the tile sets the weight reuse"):
 *     the matrix-matrix path over 32- or 64-token tiles, and the one-token
 *     matrix-vector path;
 *   - llama.cpp pull request "metal : fix idle threads in mul_mv_iq3_xxs for
 *     ne00 < 1024" (sections "Overview" and "Additional information"): the
 *     matrix-vector path at narrow K and its expert-indexed (MUL_MAT_ID) form;
 *   - tiny-llm pull request "perf: Optimize quantized matmul for small decode
 *     batches" (section "Summary"): the matrix-vector path at 1..16 tokens.
 *
 * Conventions for every call
 * --------------------------
 *  - Pointers named "device" must point to device memory of the current HIP
 *    device; the library never dereferences them on the host.
 *  - The library never allocates or frees device memory and never synchronises.
 *    Every call that launches work is asynchronous on the given stream; a device
 *    fault surfaces at the caller's next synchronisation.
 *  - Argument checks happen before any launch.  On error nothing is launched,
 *    the call returns a negative qmm_status, and qmm_last_error() holds a
 *    thread-local description.  No C++ exception crosses this interface.
 *  - Buffers passed in (blocks, x, ids) are borrowed: they must stay alive and
 *    unmodified until the stream has passed the launched work.  y must not
 *    alias x, ids or the blocks.
 *  - A handle is immutable after qmm_create, so concurrent calls with one handle
 *    on different streams are safe.
 */
#ifndef QMM_H
#define QMM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as hipStream_t; NULL is the default stream. */
typedef struct ihipStream_t *qmm_stream_t;

/*
 * Block formats (byte layouts are this library's; the pages print none).
 * fp16 fields are little-endian IEEE binary16.  Row r of a matrix starts at byte
 * r * qmm_row_bytes(type, K); expert e of a stacked tensor at e * M * row_bytes.
 *
 *  QMM_Q4_0   32 weights / 18 B: [0,2) d | [2,18) qs[16]; weight i = low nibble of
 *             qs[i], weight i+16 = high nibble.  w = d * (q - 8).
 *  QMM_Q8_0   32 weights / 34 B: [0,2) d | [2,34) int8 q[32].  w = d * q.
 *  QMM_Q4_K   256 weights / 144 B: [0,2) d | [2,4) dmin | [4,16) 96-bit little-endian
 *             string of sixteen 6-bit fields (field f at bit 6f: sc_0..sc_7, then
 *             m_0..m_7) | [16,144) qs[128]: weight 64p+i = low nibble of qs[32p+i],
 *             weight 64p+32+i = high nibble (p = 0..3, i = 0..31).
 *             w = d * sc_j * q - dmin * m_j with j = weight / 32.
 *  QMM_Q6_K   256 weights / 210 B: [0,2) d | [2,18) int8 sc[16] | [18,146) ql[128]:
 *             weight i (< 128) low nibble of ql[i], weight i+128 high nibble |
 *             [146,210) qh[64]: bits 2b..2b+1 of qh[i] are the top two bits of
 *             weight i+64b.  q = low4 | high2 << 4.  w = d * sc_j * (q - 32), j = weight / 16.
 *  QMM_A4G64  64 weights / 36 B: [0,2) scale | [2,4) bias | [4,36) qs[32]; weight i =
 *             low nibble of qs[i], weight i+32 = high nibble.  w = scale * q + bias.
 *
 * The other types the candle pull request lists (section "What changes"); the
 * pages give no formula for them, so they are read from their names ("_0": a
 * scale times a zero-centred code, "_1": a scale and a minimum, K-quants:
 * 256-weight super-blocks with per-sub-block scales and minimums):
 *  QMM_Q4_1   32 weights / 20 B: [0,2) d | [2,4) m | [4,20) qs[16] as Q4_0.  w = d * q + m.
 *  QMM_Q5_0   32 weights / 22 B: [0,2) d | [2,6) qh, 32-bit little-endian, bit i the top
 *             (fifth) bit of weight i | [6,22) qs[16], low nibbles as Q4_0.  w = d * (q - 16).
 *  QMM_Q5_1   32 weights / 24 B: [0,2) d | [2,4) m | [4,8) qh | [8,24) qs[16] as Q5_0.
 *             w = d * q + m.
 *  QMM_Q2_K   256 weights / 84 B: [0,2) d | [2,4) dmin | [4,20) sm[16]: sc_j low nibble,
 *             m_j high nibble of sm[j] | [20,84) qs[64]: weight i is bits 2(i/64)..+1 of
 *             qs[i % 64].  w = d * sc_j * q - dmin * m_j with j = weight / 16.
 *  QMM_Q3_K   256 weights / 110 B: [0,2) d | [2,14) 96-bit string of sixteen 6-bit s_j |
 *             [14,78) ql[64]: low two bits of weight i are bits 2(i/64)..+1 of ql[i % 64] |
 *             [78,110) qh[32]: top bit of weight i is bit i/32 of qh[i % 32].
 *             w = d * (s_j - 32) * (q - 4) with j = weight / 16.
 *  QMM_Q5_K   256 weights / 176 B: [0,2) d | [2,4) dmin | [4,16) sc/m string as Q4_K |
 *             [16,48) qh[32]: top bit of weight i is bit i/32 of qh[i % 32] | [48,176)
 *             qs[128], low nibbles as Q4_K.  w = d * sc_j * q - dmin * m_j, j = weight / 32.
 *
 * Every product in these formulas is exact in fp32, so the dequantized weight is
 * the fp32 round-to-nearest-even of the formula's exact value.
 */
typedef enum {
  QMM_Q4_0 = 0,
  QMM_Q8_0 = 1,
  QMM_Q4_K = 2,
  QMM_Q6_K = 3,
  QMM_A4G64 = 4,
  QMM_Q4_1 = 5,
  QMM_Q5_0 = 6,
  QMM_Q5_1 = 7,
  QMM_Q2_K = 8,
  QMM_Q3_K = 9,
  QMM_Q5_K = 10
} qmm_type;

/* Element type of activations (x) and of qmm_dequantize's output.  QMM_BF16 is taken by
 * the qmm_f8_*, qmm_route*, qmm_cache*, qmm_head* and qmm_attend* calls only, QMM_E4M3 as
 * the type of a cache by qmm_cache_create only. */
typedef enum { QMM_F32 = 0, QMM_F16 = 1, QMM_BF16 = 2, QMM_E4M3 = 3 } qmm_dtype;

/* Token tile of the matrix-matrix path (candle pull request, sections "What
 * changes" and "Where the 64-token tile is used"): AUTO applies
 * qmm_tile_for_tokens(N); 32 and 64 force a tile. */
typedef enum { QMM_TILE_AUTO = 0, QMM_TILE_32 = 32, QMM_TILE_64 = 64 } qmm_tile;

typedef int qmm_status;
#define QMM_OK 0
#define QMM_E_ARG (-1)    /* null pointer or invalid value */
#define QMM_E_TYPE (-2)   /* unknown qmm_type or qmm_dtype */
#define QMM_E_SHAPE (-3)  /* M, K, N, S or expert out of range */
#define QMM_E_ALIGN (-4)  /* a pointer is not aligned as required */
#define QMM_E_DEVICE (-5) /* no HIP device, or the current device is not gfx950 */
#define QMM_E_HIP (-6)    /* a HIP runtime error (text in qmm_last_error) */

typedef struct qmm_matrix qmm_matrix;

/*
 * qmm_create -- describe a quantized weight tensor: the block buffer, its format
 * and its shape, the operand every page's kernel reads (candle pull request,
 * section "Why the tile sets the weight reuse": a weight tile read from the
 * quantized blocks; llama.cpp pull request, section "Overview": rows of
 * 32-weight chunks; tiny-llm pull request, section "Benchmark setup": 4-bit
 * groups with a scale and a bias).  For the expert-indexed path the tensor is
 * the experts' matrices stacked (llama.cpp pull request, section "Additional
 * information": MUL_MAT_ID picks one expert's matrix per token and slot).
 *   out        receives the handle (host memory owned by the library; free it with
 *              qmm_destroy).
 *   type       block format.
 *   blocks     DEVICE pointer, 16-byte aligned, holding n_experts * M * row_bytes(K)
 *              bytes in the layout above.  Borrowed, not copied: it must outlive
 *              the handle and stay unmodified.
 *   n_experts  1 for a plain matrix; E for the stacked experts of qmm_gemm_id.
 *   M, K       rows and reduction length; K a positive multiple of the block's
 *              weight count (32 for the 32-weight types, 64 for A4G64, 256 for the
 *              K-quants); M >= 1; one matrix
 *              (M * row_bytes(K)) below 4 GiB.
 * Checks that the current device is gfx950 (QMM_E_DEVICE otherwise) and records it.
 */
qmm_status qmm_create(qmm_matrix **out, qmm_type type, const void *blocks,
                      int64_t n_experts, int64_t M, int64_t K);

/* qmm_destroy -- free a handle's host metadata (the blocks stay the caller's; see
 * qmm_create).  NULL is accepted.  Returns QMM_OK. */
qmm_status qmm_destroy(qmm_matrix *h);

/*
 * qmm_gemv -- matrix-vector path for 1..32 tokens (llama.cpp and tiny-llm pull
 * requests above): y[t, r] = sum_k x[t, k] * w[r, k], fp32 accumulation.
 *   h   a handle with n_experts == 1.
 *   x   DEVICE, [N, K] contiguous, element type xt (fp32 or fp16), 16-byte aligned.
 *   N   0..32; 0 launches nothing and returns QMM_OK; above 32 -> QMM_E_SHAPE.
 *   y   DEVICE, [N, M] contiguous fp32, 4-byte aligned; every element is written.
 * Lanes of each 64-wide wavefront are spread over (row, 32-weight chunk) pairs so
 * none idles at narrow K, and the token count picks a kernel instance that gives
 * no register to absent tokens.  fp16 calls of 5 to 32 tokens take the matrix cores
 * with exact products: there a token's outputs depend on its activations and K only
 * (the same bits at any token count from 5), and differ in summation order, not in
 * the weights, from the vector kernels, whose N-token outputs are the bits of N
 * one-token calls.
 */
qmm_status qmm_gemv(const qmm_matrix *h, const void *x, qmm_dtype xt, int64_t N,
                    float *y, qmm_stream_t stream);

/*
 * qmm_gemv_group -- qmm_gemv on `count` independent matrices in one call: the
 * matrix-vector product of the llama.cpp and tiny-llm pull requests above, for the
 * projections of one decode step that read no output of each other (a layer's
 * query, key and value projections; its gate and up projections).
 *   hs, xs, ys  HOST arrays of `count` entries: handle i (n_experts == 1), its
 *               activations ([N, K_i], element type xt, 16-byte aligned DEVICE
 *               pointer) and its output ([N, M_i] fp32, 4-byte aligned DEVICE
 *               pointer), as for qmm_gemv.  No output may overlap another output
 *               or any activation.  The arrays are read during the call only.
 *   N           0..32 tokens, the same for every matrix; 0 launches nothing.
 *   count       0..QMM_GEMV_GROUP_MAX.
 * Every output holds the bits qmm_gemv would give it.  At one token, matrices of
 * the same format and K share launches (up to four matrices per launch, one kernel
 * launch per such set); other matrices, and every matrix at N > 1, take a launch
 * of their own.  All arguments are checked before anything is launched; errors as
 * for qmm_gemv (QMM_E_ARG for a NULL array or a count out of range).
 */
#define QMM_GEMV_GROUP_MAX 64
qmm_status qmm_gemv_group(const qmm_matrix *const *hs, const void *const *xs, qmm_dtype xt,
                          int64_t N, float *const *ys, int count, qmm_stream_t stream);

/*
 * qmm_gemm -- matrix-matrix path for any N (candle pull request above).  Each
 * workgroup dequantizes a tile of weight rows once per K step into LDS as fp16
 * (round to nearest even of the fp32 weight) and multiplies it on the matrix
 * cores, with fp32 accumulation, by a tile of 32 or 64 tokens.
 *   x     DEVICE, [N, K] contiguous fp32 or fp16, 16-byte aligned; fp32 values are
 *         rounded to fp16 (nearest even) when staged.
 *   N     >= 0; a batch of sequences is passed flattened (N = batch * tokens).
 *         The handle's K must be below 2^22 (QMM_E_SHAPE otherwise).
 *   y     DEVICE, [N, M] fp32, 4-byte aligned.
 *   tile  QMM_TILE_AUTO, QMM_TILE_32 or QMM_TILE_64.  Results are bit-identical
 *         for either tile: every output is accumulated in the same order.
 */
qmm_status qmm_gemm(const qmm_matrix *h, const void *x, qmm_dtype xt, int64_t N,
                    float *y, qmm_tile tile, qmm_stream_t stream);

/*
 * qmm_gemm_workspace_bytes -- device bytes qmm_gemm_ws needs for N tokens on this
 * handle, with either activation type (the larger of the two needs); 0 when it
 * needs none: up to 16 tokens (K is divided among the waves of a workgroup), and
 * above when the call is not split (then qmm_gemm_ws computes exactly as qmm_gemm).
 * Also 0 for a NULL or expert handle and for N outside 1..2^24.
 */
size_t qmm_gemm_workspace_bytes(const qmm_matrix *h, int64_t N);

/*
 * qmm_gemm_ws -- qmm_gemm with a caller-owned workspace (same operation, tile
 * rule and arguments; candle pull request above).  Up to 16 tokens the K range is
 * divided among the waves of a workgroup of 16 weight rows, which sum their partial
 * products in LDS (no workspace).  Above, when N tokens make too few (row, token)
 * tiles to fill the GPU, or the GPU is filled better that way, the K range is divided
 * among more workgroups: each writes its partial products to its own [N, M] fp32 slab
 * of `ws`, and a second kernel sums the slabs in split order into y.  Either split
 * depends only on the handle's shape, N and the activation type, so the result is
 * deterministic and bit-identical for either tile; it can differ from qmm_gemm's in
 * rounding (both within the same error bound).  The staged operands are qmm_gemm's:
 * the fp16 weights and activations, so one-hot tokens give the staged weights.
 *   ws        DEVICE, 16-byte aligned, ws_bytes >= qmm_gemm_workspace_bytes(h, N)
 *             (QMM_E_ARG otherwise; may be NULL when that is 0).  Borrowed until
 *             the stream passes the call; must not alias x, y or the blocks.
 *             Concurrent calls need separate workspaces.
 */
qmm_status qmm_gemm_ws(const qmm_matrix *h, const void *x, qmm_dtype xt, int64_t N,
                       float *y, qmm_tile tile, void *ws, size_t ws_bytes,
                       qmm_stream_t stream);

/*
 * qmm_gemm_noalloc -- qmm_gemm_ws for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the same operation, arguments, tile rule, K split and results, bit for
 * bit, as qmm_gemm_ws, with the split's partial products in a scratch array the
 * library holds in device memory (QMM_NOALLOC_SCRATCH_BYTES per GPU, reserved when the
 * library's code is loaded on that GPU and kept until the process ends).  The call
 * allocates nothing, on the device or the host.
 *   x, xt, N, y, tile  as qmm_gemm.
 * Errors: as qmm_gemm, and QMM_E_SHAPE when the call's split needs more than
 * QMM_NOALLOC_SCRATCH_BYTES, i.e. qmm_gemm_workspace_bytes(h, N) above it (nothing is
 * launched; use qmm_gemm_ws or qmm_gemm).  QMM_E_HIP if the scratch's
 * device address cannot be found.
 * Every call on one GPU shares that GPU's scratch: calls that overlap in time on one
 * GPU (different streams, or host threads) race and must be serialised by the
 * caller, e.g. by issuing them on one stream.  The scratch keeps the last call's
 * partial products; each split call overwrites every element it reads.
 */
#define QMM_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
qmm_status qmm_gemm_noalloc(const qmm_matrix *h, const void *x, qmm_dtype xt, int64_t N,
                            float *y, qmm_tile tile, qmm_stream_t stream);

/*
 * qmm_gemm_id -- expert-indexed matrix-vector path (MUL_MAT_ID in the llama.cpp
 * pull request above): y[t, s, r] = sum_k x_ts[k] * w_{ids[t, s]}[r, k].
 *   h           handle with n_experts = E >= 1 (experts stacked in `blocks`).
 *   x           DEVICE, fp32 or fp16, 16-byte aligned.  x_per_slot = 1: [N, S, K],
 *               slot (t, s) reads row t*S + s.  x_per_slot = 0: [N, K], every slot
 *               of token t reads row t.
 *   N           0..32 tokens (0: no launch); S 1..64 slots per token.
 *   ids         DEVICE int32 [N, S], 4-byte aligned.  Duplicate ids are computed
 *               independently; an id outside [0, E) makes its output row all NaN.
 *   y           DEVICE fp32 [N, S, M].
 * The (token, slot) pairs are grouped by expert on the device, and each active
 * expert's rows are swept once per group of its pairs (two at a time on Q4_0 rows
 * of K = 512, more on the other paths); no host synchronisation, no device memory
 * beyond the arguments.
 */
qmm_status qmm_gemm_id(const qmm_matrix *h, const void *x, qmm_dtype xt, int64_t N,
                       int64_t S, int x_per_slot, const int32_t *ids, float *y,
                       qmm_stream_t stream);

/*
 * qmm_gemm_id_tiled -- expert-indexed matrix-matrix path for prefill-sized calls
 * (MUL_MAT_ID in the llama.cpp pull request above, on the token-tiled matrix
 * cores of the candle pull request): the same operation, arguments and NaN rule
 * as qmm_gemm_id, with qmm_gemm's arithmetic (weights staged as fp16, fp32
 * activations rounded to fp16, fp32 accumulation; bound 2e-3 * S).  Each
 * workgroup finds its expert, gathers the pairs routed to it in ascending pair
 * order, and multiplies that expert's rows by them tile by tile; each expert's
 * pairs are padded to the token tile on their own.
 *   N, S   N * S <= 2^18 (token, slot) pairs; S 1..64.  Any N >= 0.
 *   x      activation rows below 4 GiB in all.
 *   tile   QMM_TILE_AUTO (the tile rule on each expert's pair count), 32 or 64.
 *          Results are bit-identical for either tile, and every output row equals,
 *          bit for bit, qmm_gemm of its expert on its activation row.
 */
qmm_status qmm_gemm_id_tiled(const qmm_matrix *h, const void *x, qmm_dtype xt, int64_t N,
                             int64_t S, int x_per_slot, const int32_t *ids, float *y,
                             qmm_tile tile, qmm_stream_t stream);

/*
 * qmm_dequantize -- decode one expert's matrix (expert 0 for a plain matrix): the
 * per-block decode step of every path, written out.  The candle pull request
 * (section "Why the tile sets the weight reuse") decodes each weight tile once
 * into threadgroup memory before the matrix product; QMM_F16 returns exactly those
 * staged values, QMM_F32 the exact dequantized weights the matrix-vector paths
 * multiply by (llama.cpp pull request, section "Additional information", checks
 * both paths against a CPU backend working from the same weights).
 *   expert  0 .. n_experts - 1 (QMM_E_SHAPE otherwise).
 *   out     DEVICE [M, K] of type ot, 16-byte aligned, every element written.
 *           QMM_F32: the exact dequantized weights (the fp32 round-to-nearest-even
 *           of each formula above).  QMM_F16: round-to-nearest-even of those fp32
 *           values, as the matrix-matrix path stages them (an fp16 overflow gives
 *           an infinity).
 * Errors: QMM_E_ARG (NULL handle or out), QMM_E_TYPE (ot), QMM_E_ALIGN, QMM_E_DEVICE
 * (not the handle's device), QMM_E_HIP (launch).
 */
qmm_status qmm_dequantize(const qmm_matrix *h, int64_t expert, void *out, qmm_dtype ot,
                          qmm_stream_t stream);

/*
 * qmm_quantize -- encode fp32 weights into blocks of `type` on the GPU (the step
 * before the path), for Q4_0, Q8_0, Q4_K, Q6_K and A4G64 (QMM_E_TYPE for the others).  The pages quantize random weights to each type before
 * timing (candle pull request above, section "Numbers") but print no quantizer;
 * these are this library's closed forms, evaluated in fp64 on the exact fp32
 * inputs in the order written.  rne/up/down round to the nearest fp16 (ties to
 * even), the least fp16 >= the value, the greatest fp16 <= it; rha rounds half
 * away from zero:
 *   Q4_0   w* = element of largest |w| (first on a tie), d = rne(w* / -8),
 *          q = min(15, floor(w / d + 8.5)) (8 when d = 0).
 *   Q8_0   d = rne(max|w| / 127), q = clamp(rha(w / d), -127, 127) (0 when d = 0).
 *   Q4_K   per 32-weight sub-block j: lo_j = min(0, min w), hi_j = max w;
 *          dmin = up(max_j(-lo_j) / 63), m_j = clamp(ceil(-lo_j / dmin), 0, 63),
 *          span_j = hi_j + dmin * m_j, d = up(max_j(span_j / 15) / 63),
 *          sc_j = clamp(ceil(span_j / (15 d)), 0, 63),
 *          q = clamp(rha((w + dmin m_j) / (d sc_j)), 0, 15) (0 when d sc_j = 0);
 *          a zero divisor gives 0 before a ceil.
 *   Q6_K   a_j = max|w| per 16-weight sub-block, d = up(max_j a_j / 3937),
 *          sc_j = clamp(ceil(a_j / (31 d)), 0, 127),
 *          q = clamp(rha(w / (d sc_j)) + 32, 0, 63) (32 when d sc_j = 0).
 *   A4G64  bias = down(min w), scale = up((max w - bias) / 15),
 *          q = clamp(rha((w - bias) / scale), 0, 15) (0 when scale = 0).
 *   w       DEVICE fp32 [M, K] contiguous, 4-byte aligned; finite values whose
 *           scales fit fp16.
 *   blocks  DEVICE, 16-byte aligned, M * qmm_row_bytes(type, K) bytes, written in
 *           the block layout above (rows back to back).  M = 0: no launch.
 * Deterministic: the bytes depend only on w.
 */
qmm_status qmm_quantize(qmm_type type, const float *w, int64_t M, int64_t K, void *blocks,
                        qmm_stream_t stream);

/*
 * e4m3 products with one scale per block of 128
 * ---------------------------------------------
 * Both operands are 8-bit floats (e4m3: 4 exponent bits, 3 mantissa bits, largest value
 * 448, one NaN code, no infinity).  The values of a block share an fp32 scale:
 *   tokens    one scale per token and 128 consecutive values along K;
 *   weights   one scale per 128 rows x 128 values along K.
 *     s    = max(fp32(max |v| / 448), 2^-80)     over the block's values v
 *     code = the e4m3 value nearest to v / s     (ties to even, one rounding)
 * and a code stands for code * s.  A block that holds an Inf or a NaN gets the scale NaN
 * (its codes are unspecified): what is computed from it is NaN.
 * Let Kp = qmm_f8_padded(K), the next multiple of 128, and G = Kp / 128.
 *   codes of R rows     R * Kp bytes, row r at r * Kp; bytes K .. Kp-1 of a row are zero.
 *   scales of N tokens  fp32 [G][N]: group-major, so that a group's tokens are adjacent.
 *   scales of weights   fp32 [qmm_f8_padded(M) / 128][G] per expert.
 * With K a multiple of 128 the codes are a plain row-major matrix.
 *
 *   y[t, r] = sum_g sx[g, t] sw[r / 128, g] sum_{k in g} xq[t, k] wq[r, k]
 *
 * Sums are fp32 and y is rounded once to its type.  For an fp32 y a group's 128 products are
 * summed to 24 bits.  For a 16-bit y they run on the 8-bit matrix cores, twice as fast, which
 * cut each of 8 products at 2^-13 of the largest one's exponent.  Of the outputs' root mean
 * square that is 1.4e-5 on normal data and 6e-5 to 7e-5 with one channel of the tokens 300 times
 * larger; the rounding to fp16 is 2.1e-4 of it, to bf16 1.7e-3.  A caller that needs these bits
 * takes an fp32 y.  (Two blocks that both have the smallest scale may be left out of a sum: they
 * add less than 2^-135.)
 * The path and with it the order of the sums depends on the shapes only: the same call
 * gives the same bits.  Conventions are those at the top of this file; in addition every
 * call with nothing to compute (N = 0) returns QMM_OK without looking at its pointers.
 * Sizes: 0 <= N <= 2^24, 1 <= M <= 2^24, 1 <= K <= 2^22 - 128 unless said otherwise.
 *
 * Training: dx = dy W is the product of dy, quantized as tokens along M, with the
 * transposed matrix' codes (a 128 x 128 block transposes onto a block: the same codes and
 * scales, qmm_f8_transpose).  dW = dy^T x runs over the tokens: both operands are
 * quantized in groups of 128 tokens (codes_t of qmm_f8_quantize) and qmm_f8_wgrad
 * multiplies them.  Every gradient is a call.
 */
typedef struct qmm_f8_matrix qmm_f8_matrix;

/* n rounded up to a multiple of 128; 0 for n <= 0. */
int64_t qmm_f8_padded(int64_t n);

/*
 * qmm_f8_create / qmm_f8_destroy -- describe quantized weights (as qmm_create).
 *   codes   DEVICE, 16-byte aligned, n_experts * M * Kp bytes.
 *   scales  DEVICE fp32, 4-byte aligned, n_experts * (qmm_f8_padded(M) / 128) * G.
 * Both are borrowed.  They may be rewritten in stream order (qmm_f8_quantize_weight).
 *   n_experts 1 .. 8192.
 */
qmm_status qmm_f8_create(qmm_f8_matrix **out, const void *codes, const float *scales,
                         int64_t n_experts, int64_t M, int64_t K);
qmm_status qmm_f8_destroy(qmm_f8_matrix *h);

/*
 * qmm_f8_quantize -- quantize tokens, along K, along the tokens, or both in one pass.
 *   x         DEVICE [N, K] of type xt, row t at element t * ldx (ldx >= K), aligned to its
 *             elements (16-byte aligned rows are read faster).
 *   codes     DEVICE, 16-byte aligned, [N][Kp]; scales fp32 [G][N].  NULL, both: not wanted.
 *   codes_t   DEVICE, 16-byte aligned, [K][Np] with Np = qmm_f8_padded(N): the codes of the
 *             transpose, one scale per channel and 128 tokens; scales_t fp32 [Np / 128][K].
 *             NULL, both: not wanted.
 */
qmm_status qmm_f8_quantize(const void *x, qmm_dtype xt, int64_t ldx, int64_t N, int64_t K,
                           void *codes, float *scales, void *codes_t, float *scales_t,
                           qmm_stream_t stream);

/*
 * qmm_f8_quantize_weight -- quantize weights w [n_experts, M, K] (type wt, contiguous) in
 * blocks of 128 x 128: codes and scales as qmm_f8_create takes them.  codes_t / scales_t
 * (NULL, both: not wanted) receive the transposed matrices' (n_experts x K rows of
 * qmm_f8_padded(M) bytes).
 */
qmm_status qmm_f8_quantize_weight(const void *w, qmm_dtype wt, int64_t n_experts, int64_t M,
                                  int64_t K, void *codes, float *scales, void *codes_t,
                                  float *scales_t, qmm_stream_t stream);

/* qmm_f8_transpose -- codes and scales of the transposed matrices (as
 * qmm_f8_quantize_weight's codes_t, scales_t) from a handle's. */
qmm_status qmm_f8_transpose(const qmm_f8_matrix *h, void *codes_t, float *scales_t,
                            qmm_stream_t stream);

/* qmm_f8_dequantize -- one expert's weights code * s as [M, K] of type ot (as
 * qmm_dequantize; 16-bit outputs are rounded once more). */
qmm_status qmm_f8_dequantize(const qmm_f8_matrix *h, int64_t expert, void *out, qmm_dtype ot,
                             qmm_stream_t stream);

/*
 * qmm_f8_linear -- quantize the tokens and multiply: y = x W^T for N tokens.
 *   x     as qmm_f8_quantize.     y   DEVICE [N, M] of type yt, element-aligned.
 *   ws    DEVICE, 16-byte aligned, ws_bytes >= qmm_f8_linear_workspace_bytes(h, N) (may be
 *         NULL when that is 0: a few tokens are quantized inside the product's one launch).
 *         Borrowed until the stream passes the call; concurrent calls need separate ones.
 * qmm_f8_gemm -- the product alone, of tokens quantized before (several matrices that read
 * the same tokens share one qmm_f8_quantize).
 *   codes, scales  of N tokens.   ws  as above, qmm_f8_gemm_workspace_bytes(h, N).
 */
size_t qmm_f8_linear_workspace_bytes(const qmm_f8_matrix *h, int64_t N);
qmm_status qmm_f8_linear(const qmm_f8_matrix *h, const void *x, qmm_dtype xt, int64_t ldx,
                         int64_t N, void *y, qmm_dtype yt, void *ws, size_t ws_bytes,
                         qmm_stream_t stream);
size_t qmm_f8_gemm_workspace_bytes(const qmm_f8_matrix *h, int64_t N);
qmm_status qmm_f8_gemm(const qmm_f8_matrix *h, const void *codes, const float *scales,
                       int64_t N, void *y, qmm_dtype yt, void *ws, size_t ws_bytes,
                       qmm_stream_t stream);

/*
 * qmm_route_plan -- sort N * S (token, slot) pairs by expert for the calls below.
 *   ids   DEVICE int32 [N, S]: an expert 0 .. E-1; -1 is an empty slot (a dropped or padded
 *         token).  Duplicates are pairs of their own.  S 1..64, E 1..1024, N * S <= 2^22.
 *   plan  DEVICE, 16-byte aligned, qmm_route_plan_bytes(N * S, E) bytes.  Its first E + 2
 *         int32 are the pairs of each expert, of the empty slots and of the ids that name no
 *         expert; the rest is the library's.  The same ids give the same plan.
 */
size_t qmm_route_plan_bytes(int64_t pairs, int64_t E);
qmm_status qmm_route_plan(const int32_t *ids, int64_t N, int64_t S, int64_t E, void *plan,
                          size_t plan_bytes, qmm_stream_t stream);

/*
 * qmm_f8_linear_id / qmm_f8_gemm_id -- expert-indexed forms: y[t, s] = x_ts W_{ids[t, s]}^T,
 * y [N, S, M].  x_per_slot as qmm_gemm_id; x [rows, K] contiguous with rows = N * S or N, the
 * rows' codes below 4 GiB.  An empty slot's row is zeros, the row of an id that names no
 * expert all NaN.
 *   plan   qmm_route_plan of the ids with E = the handle's n_experts (<= 1024).
 *   ws     qmm_f8_linear_id_workspace_bytes(h, N, S, x_per_slot) bytes, as qmm_f8_linear.
 */
size_t qmm_f8_linear_id_workspace_bytes(const qmm_f8_matrix *h, int64_t N, int64_t S,
                                        int x_per_slot);
qmm_status qmm_f8_linear_id(const qmm_f8_matrix *h, const void *x, qmm_dtype xt, int64_t N,
                            int64_t S, int x_per_slot, const int32_t *ids, void *y,
                            qmm_dtype yt, void *ws, size_t ws_bytes, qmm_stream_t stream);
qmm_status qmm_f8_gemm_id(const qmm_f8_matrix *h, const void *codes, const float *scales,
                          int64_t N, int64_t S, int x_per_slot, const void *plan, void *y,
                          qmm_dtype yt, qmm_stream_t stream);

/*
 * qmm_f8_quantize_routed -- the transposed quantization (codes_t of qmm_f8_quantize) of the
 * pairs' rows in the plan's order, each expert's pairs padded to groups of 128 on their own.
 *   x   [rows, K] as qmm_f8_linear_id, row t at t * ldx.
 *   Np  = qmm_f8_routed_tokens(N * S, E), an upper bound that depends on the sizes only;
 *         codes_t [K][Np], scales_t fp32 [Np / 128][K].  Groups past the experts' own are not
 *         written (and not read by qmm_f8_wgrad_id).
 * qmm_f8_wgrad -- dw[M, K] = g^T x over N tokens, every element written.
 *   g_codes, g_scales  codes_t / scales_t of g [N, M];  x_codes, x_scales those of x [N, K].
 *   dw  DEVICE of type dt, element-aligned.  N = 0 writes zeros.  N <= 2^23.
 *   ws  DEVICE, 16-byte aligned, qmm_f8_wgrad_workspace_bytes(N, M, K) bytes, as qmm_f8_linear.
 * qmm_f8_wgrad_id -- dw[E, M, K], each expert over its own pairs (zeros where it has none);
 *   both operands from qmm_f8_quantize_routed with the same plan.
 */
int64_t qmm_f8_routed_tokens(int64_t pairs, int64_t E);
qmm_status qmm_f8_quantize_routed(const void *x, qmm_dtype xt, int64_t ldx, int64_t N,
                                  int64_t S, int x_per_slot, int64_t K, int64_t E,
                                  const void *plan, void *codes_t, float *scales_t,
                                  qmm_stream_t stream);
size_t qmm_f8_wgrad_workspace_bytes(int64_t N, int64_t M, int64_t K);
qmm_status qmm_f8_wgrad(const void *g_codes, const float *g_scales, const void *x_codes,
                        const float *x_scales, int64_t N, int64_t M, int64_t K, void *dw,
                        qmm_dtype dt, void *ws, size_t ws_bytes, qmm_stream_t stream);
qmm_status qmm_f8_wgrad_id(const void *g_codes, const float *g_scales, const void *x_codes,
                           const float *x_scales, int64_t N, int64_t S, int64_t M, int64_t K,
                           int64_t E, const void *plan, void *dw, qmm_dtype dt,
                           qmm_stream_t stream);

/*
 * qmm_route -- the router in front of the expert-indexed paths.  Per token t, over the E
 * logits l: p = softmax(l); the S experts of the largest logits, largest first, ties to the
 * lower index; a logit of -inf (a masked expert) or NaN is never chosen.
 *   logits   DEVICE [N, E] of type lt, contiguous.  E 1..1024, S 1..min(64, E).
 *   valid    DEVICE uint8 [N] or NULL: 0 marks a padded row, as if all its logits were -inf.
 *   normalise 0: weights are p of the chosen experts; 1: divided by their sum.
 *   ids      int32 [N, S] for qmm_gemm_id / qmm_route_plan; -1 where no expert is left.
 *   weights  fp32 [N, S]; 0 where the id is -1.
 *   counts   int32 [E + 1]: pairs of each expert; counts[E] = T, the rows with an expert.
 *   psum     fp32 [E]: sum over the rows of p.
 *   loss     fp32 [1] or NULL: the balance loss coef * sum_e f_e P_e with
 *            f_e = E counts[e] / (S T) and P_e = psum[e] / T; 0 when T = 0.
 *   ws       DEVICE, 16-byte aligned, qmm_route_workspace_bytes(N, E).
 * A row that has an expert and a NaN among its logits, or +inf as its largest, has NaN weights
 * and makes psum and loss NaN.  Sums over the tokens have a fixed order.  N = 0 writes zero
 * counts, psum and loss.
 *
 * qmm_balance_loss -- the loss from counts and psum, for a caller that adds them over several
 * micro-batches or GPUs first.
 *
 * qmm_route_backward -- dlogits [N, E] (type lt) of a scalar whose gradients are dweights
 * [N, S] (fp32; NULL: none) with respect to the weights and dloss (fp32 [1] on the DEVICE;
 * NULL: none) with respect to the loss.  f_e is a constant of the loss, from counts (the
 * summed ones, if they were summed); ids are qmm_route's.  Padded rows get zeros.
 */
size_t qmm_route_workspace_bytes(int64_t N, int64_t E);
qmm_status qmm_route(const void *logits, qmm_dtype lt, int64_t N, int64_t E, int64_t S,
                     const uint8_t *valid, int normalise, float coef, int32_t *ids,
                     float *weights, int32_t *counts, float *psum, float *loss, void *ws,
                     size_t ws_bytes, qmm_stream_t stream);
qmm_status qmm_balance_loss(const int32_t *counts, const float *psum, int64_t E, int64_t S,
                            float coef, float *loss, qmm_stream_t stream);
qmm_status qmm_route_backward(const void *logits, qmm_dtype lt, int64_t N, int64_t E, int64_t S,
                              const uint8_t *valid, int normalise, float coef,
                              const int32_t *ids, const float *dweights,
                              const int32_t *counts, const float *dloss, void *dlogits,
                              qmm_stream_t stream);

/*
 * qmm_route_combine -- out[t] = sum_s weights[t, s] y[t, s] over y [N, S, M], in fp32, slots in
 * order, rounded once to y's type (out [N, M] has it too).  weights [N, S] fp32 or of y's type
 * (wt); NULL: the plain sum, the gradient of a token row that its slots share.  A slot of weight
 * 0 adds nothing, whatever its row holds: qmm_gemm_id and qmm_gemm_id_tiled fill the row of an
 * empty slot (id -1, to which qmm_route gives the weight 0) with NaN.
 * qmm_route_combine_backward -- dy[t, s] = weights[t, s] dout[t] (fp32 product, rounded to y's
 * type) and dweights[t, s] = <y[t, s], dout[t]> (fp32 sum, rounded to wt), also where the weight
 * is 0: NaN for a NaN row.  qmm_route_backward takes no gradient of an empty slot.
 * All contiguous and element-aligned.  S 1..64.
 */
qmm_status qmm_route_combine(const void *y, qmm_dtype yt, const void *weights, qmm_dtype wt,
                             int64_t N, int64_t S, int64_t M, void *out, qmm_stream_t stream);
qmm_status qmm_route_combine_backward(const void *y, qmm_dtype yt, const void *weights,
                                      qmm_dtype wt, int64_t N, int64_t S, int64_t M,
                                      const void *dout, void *dy, void *dweights,
                                      qmm_stream_t stream);

/*
 * Between the projections of a served layer
 * -----------------------------------------
 * Norms and rotation of the query and key heads, a paged key-value cache, and attention over
 * it and over prompts.  Inputs x [T, heads, D] are given with the strides of a token and of a
 * head in elements (`q_token`, `q_head` and so on; the last axis is contiguous), so that slices
 * of one projection's output are taken as they are; outputs are contiguous.  D is a multiple of
 * 16, 16..256; T up to 2^30.  Serving: no gradients.  The calls take their arguments in a struct
 * in HOST memory, which is read during the call only.  Conventions are those at the top of this
 * file; a call with nothing to compute (T = 0, B = 0) returns QMM_OK without looking at its
 * pointers.
 *
 * qmm_head_norm_rope -- queries q [T, Hq, D] and keys k [T, H, D] (type xt; Hq or H may be 0):
 *   y = x / sqrt(mean(x^2) + eps) * w     over each head (not where the weight is NULL)
 *   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = positions[token] * inv_freq[i]
 *                                         for the pairs i of the first R columns
 *   q_weight, k_weight  DEVICE [D] of type wt, or NULL: no norm.   eps >= 0.
 *   positions  DEVICE int32 [T].   inv_freq  DEVICE fp32 [R / 2].
 *   R          a multiple of 8, 0 (no rotation; positions and inv_freq may be NULL) .. D.
 *   interleaved  0: pair i is columns i and i + R / 2; 1: columns 2 i and 2 i + 1.
 *   q_out, k_out  DEVICE, contiguous, type ot, element-aligned; may be q and k themselves
 *              where those are contiguous and of type ot.
 * Sums are fp32, angles 64-bit; one rounding to ot.  v and slots are not looked at.
 */
typedef struct {
  const void *q, *k, *v;
  const void *q_weight, *k_weight;
  const int32_t *positions;
  const float *inv_freq;
  const int32_t *slots;
  void *q_out, *k_out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  int64_t T, Hq, H, D, R;
  int32_t xt, wt, ot; /* qmm_dtype */
  int32_t interleaved;
  float eps;
} qmm_head_args;
qmm_status qmm_head_norm_rope(const qmm_head_args *a, qmm_stream_t stream);

/*
 * qmm_cache_create / qmm_cache_destroy -- describe a paged key-value cache (as qmm_create).
 *   k, v      DEVICE, 16-byte aligned, [pages][heads][page][D] of `type`: QMM_F16, QMM_BF16, or
 *             QMM_E4M3: codes with one fp32 scale per token and head,
 *               s = max(fp32(max |x| / 448), 2^-80),  code = the e4m3 value nearest to x / s
 *             (one rounding, ties to even; a head that holds an Inf or a NaN gets the scale NaN).
 *   k_scales, v_scales  DEVICE fp32, 16-byte aligned, [pages][heads][page]; NULL for 16-bit types.
 *   page      tokens of a page: a power of two, 16..4096.   pages * page <= 2^30.
 * All are borrowed; calls in stream order read and write them.
 *
 * A token's place is its slot, page * (tokens of a page) + row.  A sequence's places are a row of
 * a table int32 [B][W]: its token t lies on page table[b][t / page].  Entries past a sequence's
 * last page may hold anything: the calls may read them, and the cache's rows that they name, but
 * nothing of it reaches a result.
 */
typedef struct qmm_cache qmm_cache;
qmm_status qmm_cache_create(qmm_cache **out, void *k, void *v, float *k_scales, float *v_scales,
                            qmm_dtype type, int64_t pages, int64_t page, int64_t heads,
                            int64_t D);
qmm_status qmm_cache_destroy(qmm_cache *h);

/*
 * qmm_cache_write -- keys and values [T, heads, D] (type xt) to their slots, converted or
 * quantized on the way.
 *   slots  DEVICE int32 [T]; a negative one, or one past the last page, leaves its token out.
 *          The slots of a call are distinct: of two tokens with one slot it is not specified
 *          which is left there, nor that all parts left are of the same one.
 * qmm_cache_norm_rope_write -- qmm_head_norm_rope of q and k, then qmm_cache_write of the keys
 * (as rounded to ot) and of v [T, H, D], in one launch and with the same bits.  H and D are the
 * cache's, ot is its type unless that is e4m3; k_out is not looked at.
 * qmm_cache_read -- B sequences from the cache, packed one after another: sequence b's tokens 0,
 * 1, .. become rows starts[b] .. starts[b + 1] - 1 of k and v [total, heads, D] (type ot,
 * contiguous, element-aligned).
 *   starts  DEVICE int32 [B + 1], not decreasing.  Rows before starts[0] and from starts[B] on
 *           are left as they were.
 * A token whose table entry names no page, or that lies past the table's columns, gives NaN.
 */
typedef struct {
  const void *k, *v;
  const int32_t *slots;
  int64_t k_token, k_head, v_token, v_head;
  int64_t T;
  int32_t xt; /* qmm_dtype */
} qmm_cache_write_args;
typedef struct {
  const int32_t *table, *starts;
  void *k, *v;
  int64_t B, W, total;
  int32_t ot; /* qmm_dtype */
} qmm_cache_read_args;
qmm_status qmm_cache_write(const qmm_cache *h, const qmm_cache_write_args *a, qmm_stream_t stream);
qmm_status qmm_cache_norm_rope_write(const qmm_cache *h, const qmm_head_args *a,
                                     qmm_stream_t stream);
qmm_status qmm_cache_read(const qmm_cache *h, const qmm_cache_read_args *a, qmm_stream_t stream);

/*
 * qmm_cache_attend -- attention of one new token per sequence over the cache:
 *   out[b, h] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale q[b, h].k_t - max),
 * t over the first lengths[b] tokens of the sequence, k and v of key head h / (Hq / heads).
 *   q        DEVICE [B, Hq, D] with strides, fp16 or bf16 (qt); a 16-bit cache's own type, either
 *            with an e4m3 cache.  Hq a multiple of the cache's heads.  B up to 65535.
 *   lengths  DEVICE int32 [B]; 0 gives a row of zeros; above the table's reach W * page it counts
 *            as that.  A table entry that names no page makes the sequence's outputs NaN.
 *   max_length  the longest length, as far as the caller knows it: it decides into how many
 *            pieces a sequence is divided and nothing else.
 *   scale    positive, of the scores (1 / sqrt(D) as a rule).
 *   out      DEVICE [B, Hq, D] of type qt, contiguous, element-aligned.
 *   ws       DEVICE, 16-byte aligned, qmm_cache_attend_workspace_bytes(h, B, Hq, max_length)
 *            bytes (0 for an argument that the call refuses).  Borrowed until the stream passes the
 *            call; concurrent calls need separate ones.
 * Softmax in fp32; probabilities keep 16 bits or more; outputs are rounded once.  What the cache
 * holds past a sequence's last token has no influence, whatever it is.  A row whose scores are all
 * -inf is zeros.  An infinite value that a row sees gives it an infinity, or NaN where its
 * probability is rounded to zero; one of each sign, or a NaN, gives NaN.
 */
typedef struct {
  const void *q;
  const int32_t *table, *lengths;
  void *out, *ws;
  int64_t q_token, q_head;
  int64_t B, Hq, W, max_length;
  uint64_t ws_bytes;
  int32_t qt; /* qmm_dtype */
  float scale;
} qmm_attend_args;
size_t qmm_cache_attend_workspace_bytes(const qmm_cache *h, int64_t B, int64_t Hq,
                                        int64_t max_length);
qmm_status qmm_cache_attend(const qmm_cache *h, const qmm_attend_args *a, qmm_stream_t stream);

/*
 * qmm_attend_prompt -- attention of B packed sequences: queries q [Tq, Hq, D], keys and values
 * [Tk, H, D], all fp16 or all bf16 (dt), Hq a multiple of H.
 *   q_starts, k_starts  DEVICE int32 [B + 1], not decreasing: sequence b has the n queries from
 *            q_starts[b] and the m keys from k_starts[b] on (the same array without a prefix).
 *   causal   1: query i of n sees keys 0 .. i + m - n, so that the last query sees all keys; a
 *            query that sees none (n > m) gives zeros.  0: all of its sequence's keys.
 *   k, v     rows 16-byte aligned; a token's stride D .. 2^23 elements.
 *   scale    positive.    out  DEVICE [Tq, Hq, D], contiguous; rows of no sequence are left as they were.
 * Softmax in fp32, probabilities rounded to dt, outputs rounded once.  A key or value that a query
 * does not see changes no bit of its output, whatever it holds.  A row whose scores are all -inf is
 * zeros.  An infinite value that a row sees gives it an infinity, or NaN where its probability is
 * rounded to zero.
 */
typedef struct {
  const void *q, *k, *v;
  const int32_t *q_starts, *k_starts;
  void *out;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;
  int64_t B, Tq, Tk, Hq, H, D;
  int32_t dt; /* qmm_dtype */
  int32_t causal;
  float scale;
} qmm_prompt_args;
qmm_status qmm_attend_prompt(const qmm_prompt_args *a, qmm_stream_t stream);

/* qmm_tile_for_tokens -- 64 when a 64-token tile pads no more tokens than a
 * 32-token tile, else 32 (candle pull request, section "Where the 64-token tile
 * is used").  Host-only and pure; N < 0 returns 0. */
int qmm_tile_for_tokens(int64_t N);

/* Helpers.  qmm_row_bytes returns 0 for an unknown type or a K that is not a
 * positive multiple of the block; the block queries return 0 for an unknown type. */
size_t qmm_row_bytes(qmm_type type, int64_t K);
int qmm_block_weights(qmm_type type);
int qmm_block_bytes(qmm_type type);
const char *qmm_status_string(qmm_status s);
const char *qmm_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* QMM_H */
