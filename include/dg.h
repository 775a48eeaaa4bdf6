/*
 * dg.h - C ABI of the MI355X (gfx950) FP8 block-scaled GEMM library (libdg.so).
 *
 * The method: FP8 (E4M3) matrix multiplication with DeepSeek-V3 style
 * fine-grained scaling and two-level (promoted) FP32 accumulation, in three
 * forms - a normal GEMM, a contiguous-grouped MoE GEMM and a masked-grouped
 * MoE GEMM.  Beside them (end of this file): expert routing, the expert row
 * layout with dispatch and combine, the three forms in 8-bit integers, and the
 * gated feed-forward product, activation and residual norms.
 * Sources (DeepGEMM news/blog pages):
 *   - 机器之心 DeepGEMM report, opening section: fine-grained scaling as in
 *     DeepSeek-V3; normal and MoE grouped GEMMs; two-level accumulation on
 *     the general-purpose cores because FP8 tensor-core accumulation is
 *     imprecise.  Same report, "quick start": the three GEMM forms.
 *   - ai.abqq.net summary, section 3 "core functions and features": E4M3
 *     data (4-bit exponent, 3-bit mantissa); contiguous and masked layouts.
 *   - 3loumao explainer, section 03 "how DeepSeek innovated": the contiguous
 *     layout joins every expert's rows into one block; the masked layout marks
 *     which rows to compute and skips the rest at run time.
 *   - CSDN "DeepGEMM: concise, efficient ..." article, "utilities": maximum
 *     number of compute units used, the contiguous-layout alignment, and the
 *     aligned column-major activation-scale tensor.
 *
 * Conventions shared by every entry point:
 *   - All data pointers are DEVICE pointers owned by the caller; the library
 *     keeps none of them after it returns.  All pointers must be 16-byte
 *     aligned.
 *   - E4M3 means the OCP E4M3FN encoding (largest finite value 448).  FP8
 *     operands are passed as uint8_t bytes; bf16 outputs as uint16_t bits.
 *   - K (the reduction length) must be a positive multiple of 16 (16-byte rows).
 *     KB = ceil(K / 128) scale groups cover it; when K % 128 != 0 the last group
 *     holds the K % 128 elements present, its scale is their amax / 448, and the
 *     GEMM treats the absent positions as zeros (the pages ask for irregular
 *     shapes - ai.abqq.net summary, section 1 - without fixing this case).
 *   - Activation scales `sa` are stored K-group-major ("MN-major"):
 *     sa[kb * ld_sa + row] is the scale of row `row`, columns
 *     [128*kb, min(128*kb+128, K)).  ld_sa >= rows and ld_sa % 4 == 0
 *     (dg_get_scale_ld gives the smallest such value).
 *   - Weight scales `sb` are stored block-row-major: sb[nb * KB + kb] is the
 *     scale of rows [128*nb, 128*nb+128) (a partial last block is allowed),
 *     columns [128*kb, min(128*kb+128, K)).
 *   - Work is enqueued on `stream` (a hipStream_t; NULL = the default
 *     stream) without any host synchronisation: device-resident counts
 *     (m_indices, masked_m) are read by the kernels only.
 *   - Return value: DG_OK, or a negative dg_status.  Argument errors are
 *     detected synchronously, before anything is launched.  A failed launch
 *     returns DG_ERR_HIP.  Faults inside a kernel surface at the caller's next
 *     synchronisation.  A zero-sized problem (m == 0, num_groups == 0) is a
 *     successful no-op.  No C++ exception crosses this interface.
 *   - Entry points are reentrant; dg_set_num_cus is process-wide.
 */
#ifndef DG_H_
#define DG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* dg_stream_t; /* hipStream_t */

enum dg_status {
  DG_OK = 0,
  DG_ERR_INVALID_ARG = -1, /* a pointer, size, stride or alignment is invalid */
  DG_ERR_UNSUPPORTED = -2, /* valid but outside what the kernels implement */
  DG_ERR_WORKSPACE = -3,   /* workspace too small where one is required (the GEMMs that take an
                              optional workspace skip split-K instead) */
  DG_ERR_HIP = -4          /* a HIP runtime call failed */
};

/* Human-readable name of a status code (static string). */
const char* dg_status_string(int status);

/* Detail of the last non-OK return on the calling thread (thread-local, static storage). */
const char* dg_last_error_message(void);

/*
 * Per-token-group activation quantizer (1 x 128), for num_groups stacked (m, k)
 * matrices (num_groups = 1 for a plain activation matrix; the masked MoE layout
 * uses one group per expert).
 * Fine-grained scaling as in DeepSeek-V3 (机器之心 report, opening section),
 * E4M3 data (ai.abqq.net summary, section 3).  For each row r and K group kb:
 *   amax = max |x[r, 128kb .. 128kb+127]|
 *   s    = amax / 448 (IEEE fp32 division; s = 1 when amax == 0)
 *   q    = E4M3 round-to-nearest-even, saturating, of fl32(x / s) (IEEE division)
 * x  : fp32 (num_groups, m, k) row-major, read only.
 * q  : E4M3 bytes (num_groups, m, k) row-major, written.
 * sa : fp32 scales, MN-major per group: written at sa[(g * KB + kb) * ld_sa + r]
 *      for r < m; entries r >= m are untouched.
 * Errors: DG_ERR_INVALID_ARG for null/misaligned pointers, m < 0, num_groups < 0,
 * k % 16 != 0, ld_sa < m or ld_sa % 4 != 0.  Output is bit-exact (the result is unique).
 */
int dg_quantize_per_token_group(const float* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* q,
                                float* sa, int64_t ld_sa, dg_stream_t stream);

/*
 * The same per-token-group quantizer for bf16 activations (x : bf16 bits, (num_groups,
 * m, k) row-major).  A bf16 value widens to fp32 exactly, so the bytes and scales are those
 * dg_quantize_per_token_group gives for the widened values.  Activations of this path are
 * commonly bf16 (the GEMM's own output format: 机器之心 report, "quick start"); reading them
 * directly halves the quantizer's input traffic (2 B instead of 4 B per element).
 * Same layouts, errors and guarantees as dg_quantize_per_token_group.
 */
int dg_quantize_per_token_group_bf16(const uint16_t* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* q,
                                     float* sa, int64_t ld_sa, dg_stream_t stream);

/*
 * Per-block weight quantizer (128 x 128), for num_groups stacked (n, k) matrices.
 * Same rule as above with the amax over each 128 x 128 block (a partial last
 * block at the N edge takes its amax over the rows present).
 * w  : fp32 (num_groups, n, k) row-major, read only.
 * q  : E4M3 bytes (num_groups, n, k), written.
 * sb : fp32 (num_groups, ceil(n/128), KB), written.
 * Errors: DG_ERR_INVALID_ARG for null/misaligned pointers, n < 0, num_groups < 0,
 * k % 16 != 0.  Output is bit-exact.
 */
int dg_quantize_per_block(const float* w, int64_t num_groups, int64_t n, int64_t k, uint8_t* q,
                          float* sb, dg_stream_t stream);

/*
 * Normal FP8 GEMM  D = A * B^T  with two-level accumulation (机器之心 report,
 * opening section and "quick start"; 3loumao explainer, section 03).
 * After every 128-deep K block the MFMA partial P is promoted into FP32
 * accumulators:  acc += P * fl32(sa[row, kb] * sb[n/128, kb]);  D = bf16_rne(acc).
 * a  : E4M3 (m, k) row-major.        sa : fp32, MN-major with stride ld_sa (see above).
 * b  : E4M3 (n, k) row-major.        sb : fp32 (ceil(n/128), KB).
 * d  : bf16 (m, n) row-major, written.
 * workspace : optional device scratch for K splits: every tile of a small-m shape, or the
 *   tiles of a large shape's partial last round of the persistent grid (long K only).
 *   Its first 64 KiB hold per-tile arrival counters: they must be zero before the first
 *   use (e.g. a zero-filled allocation), and every call leaves them zero; the
 *   rest holds fp32 partials.  Calls sharing one workspace must be ordered on
 *   one stream (concurrent calls race).  NULL or too small (see
 *   dg_gemm_workspace_size) => no split: still correct, slower (the rounding of
 *   the split tiles' outputs may differ in the last bit: partials are summed in
 *   fixed split order).
 * Errors: DG_ERR_INVALID_ARG for null/misaligned pointers, negative sizes,
 * k % 16 != 0, ld_sa < m or ld_sa % 4 != 0.  Deterministic: the same inputs
 * give bit-identical outputs.
 */
int dg_gemm_fp8_nt(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                   const float* sb, uint16_t* d, int64_t m, int64_t n, int64_t k, void* workspace,
                   size_t workspace_bytes, dg_stream_t stream);

/*
 * Normal FP8 GEMM on unquantized activations: D = A * B^T where A, sa are the per-token-group
 * quantization of x (the rule of dg_quantize_per_token_group: 机器之心 report, opening section;
 * ai.abqq.net summary, section 3), computed inside the GEMM launch instead of by a launch of
 * its own.  The pages leave where the quantization runs open; the result is defined by the
 * two steps it replaces.
 * x  : fp32 (dg_gemm_fp8_nt_act_quant) or bf16 bits (..._bf16), (m, k) row-major, read only.
 * b, sb, d, m, n, k : as dg_gemm_fp8_nt.
 * workspace : required, at least dg_gemm_fp8_nt_act_quant_workspace_size(m, n, k) bytes.  It
 *   holds the counters (its first 64 KiB: zero before the first use, e.g. a zero-filled
 *   allocation, and left zero by every call), the quantized activations and their scales, and
 *   the split-K partials.  Calls sharing one workspace must be ordered on one stream
 *   (concurrent calls race); x and d must not overlap it.  The workgroups of one call wait
 *   for each other once (after the quantization); that wait is bounded, so counters that
 *   are not zero on entry (a misuse of the workspace) give a wrong result, not a hang.
 * Performance: on MI355X this form is slower than the two launches it replaces (the wait
 *   across all workgroups costs more than a kernel boundary); it serves callers that need
 *   a single launch.
 * Result: bit-identical to dg_quantize_per_token_group(_bf16) of x (ld_sa = dg_get_scale_ld(m))
 *   followed by dg_gemm_fp8_nt with a workspace of at least dg_gemm_workspace_size(m, n, k, 1)
 *   bytes (the same tile plan and K split).
 * Errors: DG_ERR_INVALID_ARG for null/misaligned pointers (16 bytes), negative sizes,
 * k % 16 != 0; DG_ERR_WORKSPACE when the workspace is smaller than required;
 * DG_ERR_UNSUPPORTED when m * k or n * k reaches 2^31.  Deterministic.
 */
int dg_gemm_fp8_nt_act_quant(const float* x, const uint8_t* b, const float* sb, uint16_t* d, int64_t m, int64_t n,
                             int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream);
int dg_gemm_fp8_nt_act_quant_bf16(const uint16_t* x, const uint8_t* b, const float* sb, uint16_t* d, int64_t m,
                                  int64_t n, int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream);

/*
 * The normal GEMM for callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation.  Same operation, arguments, layouts and
 * result as dg_gemm_fp8_nt (the same tile plan and K split as with a large enough workspace, so
 * the output is bit-identical to it), but the split-K counters and partials live in scratch
 * memory the library holds itself: DG_NO_ALLOC_SCRATCH_BYTES of device memory per GPU it runs
 * on, from the first call on that GPU until the process ends.  The call allocates nothing
 * (no hipMalloc, no allocating library routine).
 * Every call on one GPU shares that GPU's scratch: calls must be ordered on one stream (calls
 * that overlap on one GPU race).  The counters are cleared on the first call on a GPU (a fill
 * kernel on `stream`) and every call leaves them zero.
 * Errors: as dg_gemm_fp8_nt, plus DG_ERR_WORKSPACE (before any launch) when the plan of the
 * shape needs more scratch than DG_NO_ALLOC_SCRATCH_BYTES (no DeepSeek-V3 shape does on 256 CUs);
 * DG_ERR_HIP if the scratch address cannot be obtained.
 */
#define DG_NO_ALLOC_SCRATCH_BYTES ((size_t)64 << 20)
int dg_gemm_fp8_nt_no_alloc(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                            uint16_t* d, int64_t m, int64_t n, int64_t k, dg_stream_t stream);

/* Workspace bytes dg_gemm_fp8_nt_act_quant(_bf16) needs for a shape (0 for invalid sizes). */
size_t dg_gemm_fp8_nt_act_quant_workspace_size(int64_t m, int64_t n, int64_t k);

/*
 * Contiguous-grouped MoE GEMM (3loumao explainer, section 03: every expert's
 * rows joined into one block; ai.abqq.net summary, section 3).
 * Rows of A are grouped in blocks of dg_get_m_alignment_for_contiguous_layout()
 * (128) rows; every row of one block carries the same expert index
 * m_indices[row] in [0, num_groups).  Row r of D is A[r] * B[m_indices[r]]^T.
 * A block whose index is outside [0, num_groups) (e.g. -1 padding) is skipped
 * and its D rows are left unwritten.
 * a  : E4M3 (m_total, k);  sa : fp32 MN-major, stride ld_sa >= m_total.
 * b  : E4M3 (num_groups, n, k);  sb : fp32 (num_groups, ceil(n/128), KB).
 * m_indices : int32 (m_total,), DEVICE memory, read by the kernel only.
 * d  : bf16 (m_total, n).
 * Errors: as dg_gemm_fp8_nt, plus m_total % 128 != 0.
 */
int dg_gemm_fp8_grouped_contiguous(const uint8_t* a, const float* sa, int64_t ld_sa,
                                   const uint8_t* b, const float* sb, const int32_t* m_indices,
                                   int64_t num_groups, uint16_t* d, int64_t m_total, int64_t n,
                                   int64_t k, dg_stream_t stream);

/*
 * Masked-grouped MoE GEMM (3loumao explainer, section 03: mark which rows to
 * compute and skip invalid work such as empty decode tokens at run time).
 * For expert g only rows r < min(max(masked_m[g], 0), m_max) are computed and
 * written; rows at or past that count are never written.
 * a  : E4M3 (num_groups, m_max, k);  sa : fp32 (num_groups, KB, ld_sa), ld_sa >= m_max.
 * b  : E4M3 (num_groups, n, k);      sb : fp32 (num_groups, ceil(n/128), KB).
 * d  : bf16 (num_groups, m_max, n).
 * masked_m : int32 (num_groups,), DEVICE memory, read by the kernel only.
 * workspace : as dg_gemm_fp8_nt (used for split-K when m_max is small).
 * Errors: as dg_gemm_fp8_nt.
 */
int dg_gemm_fp8_grouped_masked(const uint8_t* a, const float* sa, int64_t ld_sa,
                               const uint8_t* b, const float* sb, uint16_t* d,
                               const int32_t* masked_m, int64_t num_groups, int64_t m_max,
                               int64_t n, int64_t k, void* workspace, size_t workspace_bytes,
                               dg_stream_t stream);

/*
 * Training-side layouts: the backward GEMMs of a linear layer Y = X * W^T.  The pages say the
 * library serves DeepSeek-V3/R1 training as well as inference (机器之心 report, opening section;
 * 3loumao explainer, section 03; ai.abqq.net summary, section 3 "application scenarios") but
 * describe no backward pass.  These entry points keep the fine-grained recipe with the scale
 * groups along each backward GEMM's own contraction dimension:
 *   dgrad  dX = dY * W       = dg_gemm_fp8_nt(dY per-token groups, W^T blocks)
 *          (W^T's 128 x 128 block quantization is W's transposed: dg_transpose_blocks);
 *   wgrad  dW = dY^T * X     = dg_gemm_fp8_nt_row_scaled(dY^T, X^T), both operands in
 *          groups of 128 tokens per column (dg_quantize_per_channel_group);
 *          per expert over the contiguous MoE layout: dg_gemm_fp8_k_grouped_row_scaled.
 */

/*
 * Per-channel-group quantizer (128 x 1: 128 consecutive tokens of one column), transposed
 * output, for num_groups stacked (m, k) matrices.  Same rule as the per-token quantizer with
 * the amax over x[128mb .. 128mb+127, col] (a last group of m % 128 tokens takes its amax over
 * the tokens present).
 * x  : fp32 (num_groups, m, k) row-major, read only.
 * qt : E4M3 bytes (num_groups, k, m) row-major, written: qt[g, col, tok] encodes x[g, tok, col].
 * st : fp32 scales in the activation-scale layout of the transposed matrix: written at
 *      st[(g * MB + mb) * ld_st + col] for col < k, MB = ceil(m / 128); other entries untouched.
 * Errors: DG_ERR_INVALID_ARG for null/misaligned pointers, negative sizes, m % 16 != 0,
 * k % 4 != 0, ld_st < k or ld_st % 4 != 0.  Output is bit-exact.
 */
int dg_quantize_per_channel_group(const float* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* qt, float* st,
                                  int64_t ld_st, dg_stream_t stream);

/* The per-channel-group quantizer for bf16 input (exact widening, as
 * dg_quantize_per_token_group_bf16).  Same layouts, errors and guarantees. */
int dg_quantize_per_channel_group_bf16(const uint16_t* x, int64_t num_groups, int64_t m, int64_t k, uint8_t* qt,
                                       float* st, int64_t ld_st, dg_stream_t stream);

/*
 * Transpose of block-quantized matrices: codes q (num_groups, rows, cols) -> qt (num_groups,
 * cols, rows), block scales s (num_groups, ceil(rows/128), ceil(cols/128)) -> st (num_groups,
 * ceil(cols/128), ceil(rows/128)).  A 128 x 128 block is square, so (qt, st) is exactly what
 * dg_quantize_per_block gives for the transposed matrix: the weight operand of the dgrad GEMM.
 * Errors: DG_ERR_INVALID_ARG for null/misaligned code pointers, negative sizes, rows or cols not
 * a multiple of 16, q == qt (no in-place transpose).  Bit-exact.
 */
int dg_transpose_blocks(const uint8_t* q, const float* s, int64_t num_groups, int64_t rows, int64_t cols, uint8_t* qt,
                        float* st, dg_stream_t stream);

/*
 * FP8 GEMM D = A * B^T where both operands carry per-row group scales (the weight-gradient
 * GEMM): after every 128-deep K block, acc += P * fl32(sa[row, kb] * sb[col, kb]);
 * D = bf16_rne(acc).
 * a  : E4M3 (m, k) row-major.   sa : fp32, sa[kb * ld_sa + row], ld_sa >= m.
 * b  : E4M3 (n, k) row-major.   sb : fp32, sb[kb * ld_sb + col], ld_sb >= n.
 * d  : bf16 (m, n) row-major, written.
 * workspace : as dg_gemm_fp8_nt (dg_gemm_workspace_size covers this form too).
 * Errors: as dg_gemm_fp8_nt, plus ld_sb < n or ld_sb % 4 != 0.  Deterministic.
 */
int dg_gemm_fp8_nt_row_scaled(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                              const float* sb, int64_t ld_sb, uint16_t* d, int64_t m, int64_t n, int64_t k,
                              void* workspace, size_t workspace_bytes, dg_stream_t stream);

/*
 * MoE weight gradients over the contiguous layout (the layout the pages name for MoE training
 * forward: 3loumao explainer, section 03): expert g's tokens are columns [start_g, start_g + T_g)
 * of both operands, start_g = T_0 + ... + T_{g-1}, and D[g] = A_g * B_g^T with per-row group
 * scales on both (dW_g = dY_g^T X_g from dg_quantize_per_channel_group of the whole dY and X:
 * every T_g is a multiple of 128, so no 128-token group straddles two experts).
 * a  : E4M3 (m, tokens_total) row-major;  sa : fp32 sa[tb * ld_sa + row], tb = token group.
 * b  : E4M3 (n, tokens_total) row-major;  sb : fp32 sb[tb * ld_sb + col].
 * d  : bf16 (num_groups, m, n), written; an expert with T_g = 0 gets zeros.
 * group_tokens : int64 (num_groups,), HOST memory, each a multiple of 128, summing to tokens_total.
 * workspace : as dg_gemm_fp8_nt, shared by the experts' GEMMs (run in order on `stream`).
 * Errors: DG_ERR_INVALID_ARG for null/misaligned pointers, negative sizes, a count that is not a
 * multiple of 128, counts not summing to tokens_total, ld_sa < m, ld_sb < n, m * n % 8 != 0.
 */
int dg_gemm_fp8_k_grouped_row_scaled(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b,
                                     const float* sb, int64_t ld_sb, uint16_t* d, const int64_t* group_tokens,
                                     int64_t num_groups, int64_t m, int64_t n, int64_t tokens_total, void* workspace,
                                     size_t workspace_bytes, dg_stream_t stream);

/*
 * Element types of the entry points below that take more than one.
 */
enum dg_dtype { DG_DTYPE_F32 = 0, DG_DTYPE_BF16 = 1, DG_DTYPE_F16 = 2 };

/*
 * Expert routing and the expert row layout: what lies between a router's logits and the grouped
 * GEMMs of the MoE forms above, and between their results and the tokens.  Arrays of indices,
 * weights, scales and logits need their elements' alignment only; row data (x, q, out, y, ...) the
 * 16-byte alignment of every other pointer.  Deterministic: the same inputs give the same bits.
 */

/*
 * Choice of top_k experts for each token from its logits x (tokens, experts).
 *   scores   s_i = softmax(x)_i or 1 / (1 + exp(-x_i));  a logit of -inf switches its expert off;
 *   choice   c_i = s_i + bias_i (bias: fp32 (experts,), NULL for none; it decides the choice only,
 *            the balance correction of DeepSeek-V3 style routers).  For softmax scores without bias
 *            and with group_top = 1 the logits themselves are compared (the same order);
 *   groups   num_groups groups of experts / num_groups consecutive experts; a group's value is the sum
 *            of its group_top (1 or 2) best choice values, the topk_groups best groups stay;
 *   ids      int32 (tokens, top_k): the best choices of those groups, best first; ties go to the lower
 *            expert (group); -1 where fewer than top_k experts are available;
 *   weights  fp32 (tokens, top_k): scale * s, or with renormalize scale * s / (sum of the chosen s);
 *            0 for id -1, and 0 where that sum is 0.
 * All in fp32.  A NaN logit is never chosen and makes the weights of its token's choices NaN.
 * logits : `dtype`, rows ld elements apart (ld >= experts), read only.
 * Errors: DG_ERR_INVALID_ARG for null pointers, misaligned elements, sizes outside 1 <= experts <= 1024,
 * 1 <= top_k <= min(64, experts), 1 <= topk_groups <= num_groups <= 64, experts % num_groups != 0,
 * group_top not 1 or 2, an unknown score or dtype.  tokens = 0 is a no-op.
 */
enum dg_moe_score { DG_MOE_SOFTMAX = 0, DG_MOE_SIGMOID = 1 };
int dg_moe_route(const void* logits, int dtype, int64_t ld, const float* bias, int64_t tokens, int64_t experts,
                 int64_t top_k, int64_t num_groups, int64_t topk_groups, int group_top, int score, int renormalize,
                 float scale, int32_t* ids, float* weights, dg_stream_t stream);

/*
 * Gradient of the weights of dg_moe_route with respect to the logits, the choice (ids) held fixed:
 * dlogits (tokens, experts), rows ld_out apart, written whole (0 for experts that do not matter), in
 * the logits' type, from dweights fp32 (tokens, top_k).  Entries of ids outside [0, experts) count as
 * not chosen.  Same errors as dg_moe_route.
 */
int dg_moe_route_grad(const float* dweights, const void* logits, int dtype, int64_t ld, const int32_t* ids,
                      int64_t tokens, int64_t experts, int64_t top_k, int score, int renormalize, float scale,
                      void* dlogits, int64_t ld_out, dg_stream_t stream);

/* Rows that the contiguous layout of any choice of experts fits in (a multiple of 128). */
int64_t dg_moe_layout_rows(int64_t tokens, int64_t top_k, int64_t experts);

/* Workspace bytes of dg_moe_layout (no initial content needed; 0: none). */
size_t dg_moe_layout_workspace_size(int64_t tokens, int64_t top_k, int64_t experts);

/*
 * Places the (token, k) entries of ids (int32 (tokens, top_k)) into the experts' rows, each expert's in
 * the order of token * top_k + k; ids outside [0, experts) get no row.
 *   rows_per_expert = 0: the contiguous layout of dg_gemm_*_grouped_contiguous: each expert's rows start
 *     at a multiple of 128.  m_indices int32 (rows_total,): the rows' expert, padding rows included, -1
 *     past the last expert's.  rows_total: a multiple of 128, at least dg_moe_layout_rows(...).
 *   rows_per_expert > 0: the masked layout of dg_gemm_*_grouped_masked: expert e's rows start at
 *     e * rows_per_expert; entries past its rows are dropped.  m_indices is NULL and rows_total =
 *     experts * rows_per_expert.  counts serve as masked_m.
 *   rows int32 (tokens, top_k): each entry's row, -1 for none.  sources int32 (rows_total,): each row's
 *     entry (token * top_k + k), -1 for none.  counts int32 (experts,): each expert's entries, dropped ones
 *     included.
 * workspace : at least dg_moe_layout_workspace_size bytes; calls that share it must be ordered.
 * Errors: DG_ERR_INVALID_ARG as above, for experts outside [1, 1024] and top_k outside [1, 64];
 * DG_ERR_WORKSPACE; DG_ERR_UNSUPPORTED for 2^31 entries or rows.
 */
int dg_moe_layout(const int32_t* ids, int64_t tokens, int64_t top_k, int64_t experts, int64_t rows_per_expert,
                  int64_t rows_total, int32_t* rows, int32_t* sources, int32_t* m_indices, int32_t* counts,
                  void* workspace, size_t workspace_bytes, dg_stream_t stream);

/*
 * Copies each token's row of x (tokens, hidden) to the rows of its entries in a layout (its rows,
 * sources, m_indices, rows_total, rows_per_expert).  In the contiguous layout the padding rows of every
 * expert are written as zeros (their scales as 1); rows of no expert, and the masked layout's rows past
 * an expert's count, stay untouched.
 *   dg_moe_dispatch       out: (rows_total, hidden) in x's type;
 *   dg_moe_dispatch_fp8   q: E4M3 bytes, sa: the activation scales of dg_quantize_per_token_group for the
 *                         same matrices (contiguous: sa[kb * ld_sa + row]; masked: per expert), bit for bit
 *                         (a NaN does not take part in its group's amax unless the group holds only NaNs);
 *   dg_moe_dispatch_int8  q, s: as dg_quantize_int8_per_token gives them, s fp32 (rows_total,).
 * workspace (FP8) : optional, dg_moe_dispatch_fp8_workspace_size bytes of any content (0: none is used);
 *   without it the same bits, slower where there are many scales.  Calls that share it must be ordered.
 * The gradient with respect to x is dg_moe_combine of the rows' gradients without weights.
 * Errors: DG_ERR_INVALID_ARG as above, hidden not a positive multiple of 16, ld_sa too small or not a
 * multiple of 4.
 */
int dg_moe_dispatch(const void* x, int dtype, const int32_t* rows, const int32_t* sources, const int32_t* m_indices,
                    int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total, int64_t rows_per_expert,
                    void* out, dg_stream_t stream);
int dg_moe_dispatch_fp8(const void* x, int dtype, const int32_t* rows, const int32_t* sources, const int32_t* m_indices,
                        int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total, int64_t rows_per_expert,
                        uint8_t* q, float* sa, int64_t ld_sa, void* workspace, size_t workspace_bytes,
                        dg_stream_t stream);
size_t dg_moe_dispatch_fp8_workspace_size(int64_t tokens, int64_t top_k, int64_t hidden);
int dg_moe_dispatch_int8(const void* x, int dtype, const int32_t* rows, const int32_t* sources,
                         const int32_t* m_indices, int64_t tokens, int64_t top_k, int64_t hidden, int64_t rows_total,
                         int64_t rows_per_expert, int8_t* q, float* s, dg_stream_t stream);

/*
 * y[t] = sum over k of weights[t, k] * out[rows[t, k]] (entries without a row add nothing; weights NULL:
 * all 1), in fp32 in the order of k, rounded once.  out (rows_total, hidden), y (tokens, hidden) in `dtype`.
 */
int dg_moe_combine(const void* out, int dtype, const int32_t* rows, const float* weights, int64_t tokens, int64_t top_k,
                   int64_t hidden, int64_t rows_total, void* y, dg_stream_t stream);

/*
 * Gradients of the weighted combine: dout[rows[t, k]] = weights[t, k] * dy[t] (padding rows of the
 * contiguous layout 0, other rows untouched) and dweights[t, k] = <dy[t], out[rows[t, k]]> in fp32 (0 for
 * entries without a row).
 */
int dg_moe_combine_grad(const void* dy, const void* out, int dtype, const int32_t* rows, const int32_t* sources,
                        const int32_t* m_indices, const float* weights, int64_t tokens, int64_t top_k, int64_t hidden,
                        int64_t rows_total, void* dout, float* dweights, dg_stream_t stream);

/*
 * 8-bit integer GEMMs: D = (A * B^T) * sa[row] * sb[col] with one fp32 scale per token (row of A) and
 * one per output channel (row of B).  The sum over K is exact in int32; scales (in an order in which their own
 * product's range is no limit) and the one rounding to the output's type (out_dtype, a dg_dtype) follow it.  K is a
 * multiple of 16 as everywhere, and at most 131056 (what int32 holds of products of any codes);
 * DG_ERR_UNSUPPORTED above.
 */

/*
 * Per-row quantizer: s = amax / 127 over the row (1 when amax = 0), q = rne(x / s) saturated to
 * [-127, 127], both IEEE fp32 divisions.  x (rows, k) in `dtype` - activations (a scale per token) or weights
 * (a scale per output channel); q int8 (rows, k); s fp32 (rows,).  Bit-exact, also where amax / 127 is
 * subnormal (fp32 rows of amax below 1.5e-36; it is 0 for amax of 63 * 2^-149 and less).  A row with a NaN or
 * an infinity gets a NaN or infinite scale (its product is NaN).
 */
int dg_quantize_int8_per_token(const void* x, int dtype, int64_t rows, int64_t k, int8_t* q, float* s,
                               dg_stream_t stream);

/*
 * Normal form: a (m, k), sa (m,), b (n, k), sb (n,), d (m, n).
 * workspace : optional, as dg_gemm_fp8_nt's (counter prefix zero before the first use, left zero); NULL
 *   or smaller than dg_gemm_int8_workspace_size(m, n, k, 1): no K split.  The result is the same bits.
 */
int dg_gemm_int8_nt(const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d, int out_dtype,
                    int64_t m, int64_t n, int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream);

/*
 * Normal form on unquantized activations x (m, k) in `dtype`: dg_quantize_int8_per_token followed by
 * dg_gemm_int8_nt, the same bits, in one call.
 * workspace : required, dg_gemm_int8_nt_act_quant_workspace_size(m, n, k) bytes, counter prefix as above (0 for
 *   one or two rows of at most 16384 elements, which need none: NULL).
 */
int dg_gemm_int8_nt_act_quant(const void* x, int dtype, const int8_t* b, const float* sb, void* d, int out_dtype,
                              int64_t m, int64_t n, int64_t k, void* workspace, size_t workspace_bytes,
                              dg_stream_t stream);
size_t dg_gemm_int8_nt_act_quant_workspace_size(int64_t m, int64_t n, int64_t k);

/* Contiguous-grouped form (layout and skipping as dg_gemm_fp8_grouped_contiguous): a (m_total, k),
 * sa (m_total,), b (num_groups, n, k), sb (num_groups, n), d (m_total, n). */
int dg_gemm_int8_grouped_contiguous(const int8_t* a, const float* sa, const int8_t* b, const float* sb,
                                    const int32_t* m_indices, int64_t num_groups, void* d, int out_dtype,
                                    int64_t m_total, int64_t n, int64_t k, dg_stream_t stream);

/* Masked-grouped form (as dg_gemm_fp8_grouped_masked): a (num_groups, m_max, k), sa (num_groups, m_max),
 * b (num_groups, n, k), sb (num_groups, n), d (num_groups, m_max, n); rows at or past masked_m[g] are
 * never written. */
int dg_gemm_int8_grouped_masked(const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* d,
                                int out_dtype, const int32_t* masked_m, int64_t num_groups, int64_t m_max, int64_t n,
                                int64_t k, void* workspace, size_t workspace_bytes, dg_stream_t stream);

/* Workspace bytes that let dg_gemm_int8_nt / dg_gemm_int8_grouped_masked split K (0: never split). */
size_t dg_gemm_int8_workspace_size(int64_t m, int64_t n, int64_t k, int64_t num_groups);

/*
 * The activation of a gated feed-forward block on its two projections, and the backward pass.
 *   pre (rows, 2n): a row holds g (n) and then u (n);  h = act(g) * u, in fp32, rounded once.
 *   DG_ACT_SILU: act(g) = g / (1 + exp(-g));  DG_ACT_GELU: the tanh form, 0.5 g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))).
 * Deterministic.  Row data needs the 16-byte alignment of every other pointer, index and scale arrays their elements'.
 * Outputs must not overlap inputs.
 */
enum dg_act { DG_ACT_SILU = 0, DG_ACT_GELU = 1 };

/*
 * Gated FP8 GEMMs: both projections of a feed-forward block, the activation and the product in one launch.
 *   g = A * Bg^T, u = A * Bu^T (each with the block scales and promoted sums of dg_gemm_fp8_nt);  h = act(g) * u in fp32.
 * a, sa   : as dg_gemm_fp8_nt (contiguous, masked: as those forms).
 * b, sb   : E4M3 (2, n, k) and fp32 (2, ceil(n/128), KB) per group: the gate matrix, then the up matrix, each quantized by
 *           itself (dg_quantize_per_block of 2 matrices per group; where n % 128 == 0 that is its result for (2n, k)).
 * output  : exactly one of
 *           d  bf16 (m, n), h rounded once, or
 *           q, s: the codes and scales that dg_quantize_per_token_group gives for h in fp32, s[nb * ld_s + row] (masked: per
 *           group), ready for the next FP8 product; n % 16 == 0, ld_s >= m (m_max), ld_s % 4 == 0.
 * pre     : bf16 (m, 2n), a row (g | u) rounded once, as dg_gated_act_grad reads it; NULL if it is not wanted.
 * Rows that the plain forms leave unwritten (m_indices outside [0, num_groups), rows at or past masked_m) are left
 * unwritten in every output.
 * workspace : as dg_gemm_fp8_nt's (its first 64 KiB zero before the first use, left zero by every call; calls that share it
 *   must be ordered); NULL or smaller than dg_gemm_fp8_gated_workspace_size: no K split.
 * Errors: as the plain forms, an unknown activation, both or neither of d and q, q without s; DG_ERR_UNSUPPORTED where 2 n k or
 * m k reaches 2^31, or KB ld_sa 2^29.  Deterministic; without a K split the g and u of a bf16 output are the bits of the
 * plain forms.
 * Precision of quantized outputs: the matrix instruction adds eight neighbouring FP8 products cut at 2^-13 of the largest's
 * power of two.  Products are exact and added in fp32 instead where the output has at most 2^19 values (m n; masked:
 * num_groups m_max n), where m (m_max) is at most 64, and for the groups of at most 64 rows of a larger masked buffer.
 * Elsewhere one or two codes in 10^4 may be the neighbours of the nearest ones to h.
 */
int dg_gemm_fp8_gated_nt(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb, int act,
                         uint16_t* d, uint8_t* q, float* s, int64_t ld_s, uint16_t* pre, int64_t m, int64_t n, int64_t k,
                         void* workspace, size_t workspace_bytes, dg_stream_t stream);
int dg_gemm_fp8_gated_contiguous(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                                 const int32_t* m_indices, int64_t num_groups, int act, uint16_t* d, uint8_t* q, float* s,
                                 int64_t ld_s, uint16_t* pre, int64_t m_total, int64_t n, int64_t k, dg_stream_t stream);
int dg_gemm_fp8_gated_masked(const uint8_t* a, const float* sa, int64_t ld_sa, const uint8_t* b, const float* sb,
                             const int32_t* masked_m, int64_t num_groups, int act, uint16_t* d, uint8_t* q, float* s,
                             int64_t ld_s, uint16_t* pre, int64_t m_max, int64_t n, int64_t k, void* workspace,
                             size_t workspace_bytes, dg_stream_t stream);

/* Workspace bytes that let dg_gemm_fp8_gated_nt / _masked split K (0: never split), and the tile and K split of a shape
 * (layout 0 normal, 1 contiguous, 2 masked), as dg_gemm_workspace_size and dg_gemm_config_name. */
size_t dg_gemm_fp8_gated_workspace_size(int64_t m, int64_t n, int64_t k, int64_t num_groups);
const char* dg_gemm_fp8_gated_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t num_groups);

/*
 * h from pre (`dtype`; n a positive multiple of 16):
 *   dg_gated_act       h (rows, n) in pre's type;
 *   dg_gated_act_fp8   q, s: the codes and scales that dg_quantize_per_token_group gives for h in fp32 (its layout of
 *                      scales: s[nb * ld_s + row]; per group with masked_m), nothing rounded before;
 *   dg_gated_act_int8  q, s: as dg_quantize_int8_per_token gives them for h in fp32, s (rows,).
 * Rows that are not computed are neither read nor written:
 *   m_indices (rows,) (not NULL): those of a negative index (the contiguous layout's padding behind the last expert);
 *   masked_m (rows / rows_per_group,) (not NULL): those at or past their group's count (the masked layout).
 * Errors: DG_ERR_INVALID_ARG for null or misaligned pointers, an unknown dtype or activation, n % 16 != 0, negative sizes, both
 * masks, masked_m without a rows_per_group that divides rows (or with one and no masked_m), ld_s too small or not a multiple
 * of 4; DG_ERR_UNSUPPORTED for shapes past the launch grid.  rows = 0 is a no-op.
 */
int dg_gated_act(const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                 int64_t rows_per_group, int64_t rows, int64_t n, void* h, dg_stream_t stream);
int dg_gated_act_fp8(const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                     int64_t rows_per_group, int64_t rows, int64_t n, uint8_t* q, float* s, int64_t ld_s,
                     dg_stream_t stream);
int dg_gated_act_int8(const void* pre, int dtype, int act, const int32_t* m_indices, const int32_t* masked_m,
                      int64_t rows_per_group, int64_t rows, int64_t n, int8_t* q, float* s, dg_stream_t stream);

/*
 * The gradient of pre: dpre (rows, 2n) = (dh * u * act'(g) | dh * act(g)), dh (rows, n) and pre in `dtype`.
 *   dg_gated_act_grad      dpre in that type; n a positive multiple of 16.
 *   dg_gated_act_grad_fp8  dpre and h as the backward FP8 products read them, from one pass over dh and pre; each pair may be
 *     NULL if it is not wanted (one must not be):
 *     q (rows, 2n), s[kb * ld_s + row]      as dg_quantize_per_token_group of dpre: the input gradient dpre * W (W^T's codes
 *                                           from dg_transpose_blocks);
 *     qt (2n, rows), st[mb * ld_st + col]   as dg_quantize_per_channel_group of dpre: the weight gradient dpre^T * X;
 *     ht (n, rows), hst[mb * ld_hst + col]  as dg_quantize_per_channel_group of h: the next product's weight gradient.
 *     n a positive multiple of 128 (the groups of q must not hold columns of both halves), rows a multiple of 16.
 * Errors: as above, and a code pointer without its scales or the reverse.
 */
int dg_gated_act_grad(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, void* dpre,
                      dg_stream_t stream);
int dg_gated_act_grad_fp8(const void* dh, const void* pre, int dtype, int act, int64_t rows, int64_t n, uint8_t* q,
                          float* s, int64_t ld_s, uint8_t* qt, float* st, int64_t ld_st, uint8_t* ht, float* hst,
                          int64_t ld_hst, dg_stream_t stream);

/*
 * What lies between two blocks of a transformer, in one pass over the rows (hidden: a multiple of 16, at most 16384):
 *   z = post_weight * x / sqrt(mean(x^2) + eps)   the norm after the first block (post_norm != 0; otherwise z = x)
 *   sum = residual + scale * gate * z             its gate and residual scale, and the residual stream
 *   y = weight * sum / sqrt(mean(sum^2) + eps)    the norm before the second block, of the sum as it is before rounding
 * All in fp32, each output rounded once; sums of squares are fp32 (values up to 1e18).
 *   x         (rows, hidden) in `dtype`, the first block's output; NULL for a norm alone (sum = residual is then not
 *             written, `sum` and `gate` are NULL and post_norm is 0);
 *   residual  (rows, hidden) in `residual_dtype`: DG_DTYPE_F32 or `dtype`;
 *   weight, post_weight  fp32 (hidden,), NULL for ones;
 *   gate      (gate_rows, hidden) in `dtype`, NULL (gate_rows 0) for none; gate_rows divides rows: gate row i serves the i-th
 *             rows / gate_rows consecutive rows (1: one gate for all; rows: each row its own);
 *   sum       (rows, hidden) in residual_dtype, NULL if it is not wanted; it may be `residual` itself (in place);
 *   y         dg_residual_norm: (rows, hidden) in `dtype`;
 *             dg_residual_norm_fp8: q, s as dg_quantize_per_token_group gives them for y in fp32;
 *             dg_residual_norm_int8: q, s as dg_quantize_int8_per_token gives them for y in fp32.
 * Errors: DG_ERR_INVALID_ARG for null or misaligned pointers, unknown types, a residual_dtype that is neither, hidden % 16 != 0,
 * gate_rows that does not divide rows, a negative or non-finite eps, ld_s too small or not a multiple of 4;
 * DG_ERR_UNSUPPORTED for hidden > 16384 or 2^31 rows.  rows = 0 is a no-op.  Deterministic.
 */
int dg_residual_norm(const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                     const void* gate, int64_t gate_rows, int post_norm, const float* post_weight, float scale, float eps,
                     int64_t rows, int64_t hidden, void* sum, void* y, dg_stream_t stream);
int dg_residual_norm_fp8(const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                         const void* gate, int64_t gate_rows, int post_norm, const float* post_weight, float scale,
                         float eps, int64_t rows, int64_t hidden, void* sum, uint8_t* q, float* s, int64_t ld_s,
                         dg_stream_t stream);
int dg_residual_norm_int8(const void* x, const void* residual, int dtype, int residual_dtype, const float* weight,
                          const void* gate, int64_t gate_rows, int post_norm, const float* post_weight, float scale,
                          float eps, int64_t rows, int64_t hidden, void* sum, int8_t* q, float* s, dg_stream_t stream);

/*
 * Gradients of dg_residual_norm from dy (rows, hidden) in `dtype`, dsum (residual_dtype; what the sum gets from elsewhere; NULL
 * for none), x (NULL as there) and sum as the forward pass stored it:
 *   dresidual (residual_dtype; it may be dsum itself) and dx (`dtype`; NULL with x), written;
 *   dweight, dpost_weight fp32 (hidden,), dgate (gate_rows, hidden) in `dtype`: written where not NULL (sums over the rows,
 *   in fp32 in a fixed order, at most 256 rows one after the other up to 2^22 of them, rounded once; NULL where there is no
 *   weight, norm or gate).
 * workspace : dg_residual_norm_grad_workspace_size(rows, hidden) bytes of any content; calls that share it must be ordered.
 *   Not needed (NULL) where dweight, dpost_weight and dgate are NULL.
 * Errors: as dg_residual_norm; DG_ERR_WORKSPACE.  rows = 0 writes zeros to the three sums.
 */
int dg_residual_norm_grad(const void* dy, const void* dsum, const void* x, const void* sum, int dtype, int residual_dtype,
                          const float* weight, const void* gate, int64_t gate_rows, int post_norm,
                          const float* post_weight, float scale, float eps, int64_t rows, int64_t hidden, void* dx,
                          void* dresidual, float* dweight, void* dgate, float* dpost_weight, void* workspace,
                          size_t workspace_bytes, dg_stream_t stream);
size_t dg_residual_norm_grad_workspace_size(int64_t rows, int64_t hidden);

/*
 * Utilities (CSDN article, "utilities": cap on the compute units used,
 * contiguous-layout alignment, aligned column-major scale tensor).
 */

/* Current cap on the compute units the persistent GEMM grid uses (default: all
 * CUs of the current device; queries the device on first use, returns < 0 on a
 * HIP error). */
int dg_get_num_cus(void);

/* Set that cap (1 <= n); n larger than the device's CU count is clamped.  Process-wide.
 * With no device visible, the cap stands in for the device's CU count in the planning
 * queries below (dg_gemm_workspace_size, dg_gemm_config_name, ...), so that plans can be
 * inspected on a host without a GPU.  Returns DG_OK or DG_ERR_INVALID_ARG. */
int dg_set_num_cus(int n);

/* Row alignment required of each group in the contiguous layout: 128. */
int dg_get_m_alignment_for_contiguous_layout(void);

/* Smallest valid ld_sa for `rows` rows: rows rounded up to a multiple of 4 (16 bytes). */
int64_t dg_get_scale_ld(int64_t rows);

/* Workspace bytes that let dg_gemm_fp8_nt / dg_gemm_fp8_nt_row_scaled /
 * dg_gemm_fp8_grouped_masked use split-K for the given shape (m = rows per group; num_groups = 1 for the
 * normal GEMM).  0 means split-K is never used for that shape. */
size_t dg_gemm_workspace_size(int64_t m, int64_t n, int64_t k, int64_t num_groups);

/* Name of the tile configuration and K split the GEMM picks for a shape, as
 * "BNxBM/Wwaves/splitS", or "BNxBM/Wwaves/split1+tailS" when only the last round's
 * tiles are split in S (static thread-local string), assuming a large enough
 * workspace.  layout: 0 normal, 1 contiguous-grouped, 2 masked-grouped (m = rows
 * per group), 3 row-scaled normal.  For profiling and reports; returns "" for invalid arguments. */
const char* dg_gemm_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t num_groups);

/* The same for the 8-bit integer GEMMs (layout 0, 1 or 2): "BNxBM/Wwaves/splitS" for tiles,
 * "stripBNxBM/Wwaves/splitS" for the kernel that streams strips of the weights past few rows.  One or two rows
 * that dg_gemm_int8_nt_act_quant quantizes itself run on a kernel without a choice of plans. */
const char* dg_gemm_int8_config_name(int layout, int64_t m, int64_t n, int64_t k, int64_t num_groups);

/*
 * Debug facility (the analogue of the pages' debug switch among the environment variables,
 * CSDN article, "environment variables").  With DG_DEBUG set to a value other than "" or "0"
 * in the environment (read at every call):
 *   - every GEMM launch logs its plan (tile configuration, K split, tiles, workspace) on stderr;
 *   - the contiguous-grouped GEMM checks m_indices on the device: each 128-row block must carry
 *     one expert index, in [0, num_groups) or -1 for the whole block.  A violation sets
 *     DG_DIAG_MIXED_BLOCK or DG_DIAG_EXPERT_RANGE; the GEMM itself proceeds as without the check
 *     (no trap, no fault: the rows of a mixed block are computed with the block's first expert).
 * Independently of DG_DEBUG, the in-launch activation quantization sets DG_DIAG_FQ_TIMEOUT when
 * its bounded wait gives up (a workspace whose counters were not zero): that call's output is
 * not valid.
 * The flags are sticky, one set per device, shared by every call on it.
 *
 * Planner override for measurement (DG_PLAN, read at every call): "tile=BNxBM" and / or
 * "splits=S", comma-separated (e.g. "tile=64x128,splits=4").  The tile replaces the planner's
 * choice when it is one the planner could pick for the form and size (64x64 or 64x128 for
 * m <= 128 rows; 256x128, 256x192 or 256x256 above; 256x128 or 256x256 for the contiguous form,
 * 256x128 for the row-scaled one); splits
 * (1..16) split every tile's K range where the call may split K.  Anything else is ignored.
 * The 8-bit integer GEMMs take "tile=256x256" or "tile=128x128", or "strip=32", 64, 96 or 128 (rows of the
 * weights; the normal and masked forms of at most 1024 rows, 96 of at most 64), and "splits=S" likewise; their
 * results stay the same bits.
 * The gated FP8 GEMMs take "tile=256x128" or "tile=256x256", or "stream=16" or 64 (rows of the streaming kernel's
 * tile; not the contiguous form), and "splits=S", to 32 for the streaming kernel.  A forced 256x128 or 256x256 tile has the
 * FP8 instruction's products where the plan's own tile would have exact ones (dg_gemm_fp8_gated_nt).  The name
 * reported is a bf16 output's plan; the workspace is enough for either output.
 * dg_gemm_config_name and dg_gemm_workspace_size (dg_gemm_int8_..., dg_gemm_fp8_gated_...) report the overridden plan; results stay within
 * the GEMM tolerance (a different K split changes the fp32 summation order).  For measuring the
 * alternatives the planner weighs, not for production use.
 */
enum dg_diag_flag {
  DG_DIAG_MIXED_BLOCK = 1,
  DG_DIAG_EXPERT_RANGE = 2,
  DG_DIAG_FQ_TIMEOUT = 4
};

/* Reads the diagnostics flags of the current device into *flags, and into *block (if not NULL)
 * the index of the first 128-row block a contiguous-layout check found wrong (-1 if none).
 * SYNCHRONISES the device first (a debugging call, not for the hot path).  clear != 0 resets
 * the flags afterwards.  Returns DG_OK, DG_ERR_INVALID_ARG (flags NULL) or DG_ERR_HIP. */
int dg_get_debug_status(uint32_t* flags, int64_t* block, int clear);

#ifdef __cplusplus
}
#endif

#endif /* DG_H_ */
