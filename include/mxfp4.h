/*
 * mxfp4.h -- MXFP4 entry points of libnvfp4.so: block quantization with power-of-two scales, its
 * expansion, the product with MXFP4 weights, a mixture-of-experts layer for a few tokens, and products whose
 * rows pick their weights (router, products grouped by expert, the layer for any number of tokens, adapters
 * per request), as hand-written HIP kernels for AMD Instinct MI355X (gfx950).
 *
 * MXFP4 (OCP Microscaling Formats, MXFP4): E2M1 codes as in nvfp4.h (magnitudes {0, 0.5, 1, 1.5, 2,
 * 3, 4, 6} and a sign bit, element 2j of a row in the low nibble of byte j), and one E8M0 byte b per
 * 32 consecutive elements of a row: value = e2m1 x 2^(b - 127); b = 255 makes the block NaN.  There
 * is no tensor scale; storage is 4.25 bits per element.  gfx950's scaled matrix instructions take
 * this format as it is stored, so MXFP4 products run at the FP4 rate of the matrix cores, which NVFP4
 * (an E4M3 scale per 16 elements) cannot.
 *
 * The conventions of nvfp4.h hold for every entry point here: caller-owned device memory, work
 * enqueued on `stream` without synchronizing, arguments validated before anything is enqueued,
 * row strides in elements, 16-byte aligned pointers and row starts except for the outputs C and y
 * (whose rows need the alignment of their element), thread-safe, capturable in a HIP graph.  No
 * workspace needs initial contents; calls that share a workspace must be ordered by the caller.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* An MXFP4 tensor of logical shape [rows x cols], cols % 32 == 0, dense:
 *   codes   rows * cols/2 bytes, row-major; element 2j of a row in the low nibble of byte j
 *   scales  rows * cols/32 bytes, row-major; E8M0                                             */
typedef struct {
    uint8_t *codes;
    uint8_t *scales;
    int64_t rows, cols;
} mxfp4_tensor;

/* Operation selectors for mxfp4_workspace_size. */
enum {
    MXFP4_OP_GEMM_BF16 = 0, /* mxfp4_gemm with bf16 activations: (M, N, K)                     */
    MXFP4_OP_GEMM_MX = 1,   /* mxfp4_gemm with MXFP4 activations: (M, N, K)                    */
    MXFP4_OP_MOE = 2,       /* mxfp4_moe: (tokens * top_k, H, I)                               */
    MXFP4_OP_ROUTE = 3,     /* mxfp4_route: (tokens, top_k, experts)                           */
    MXFP4_OP_GROUP_ROWS = 4 /* mxfp4_group_rows: (tokens, per_token, groups)                   */
};

/* Largest arguments of mxfp4_moe. */
enum { MXFP4_MOE_MAX_TOKENS = 64, MXFP4_MOE_MAX_EXPERTS = 512, MXFP4_MOE_MAX_TOP_K = 16 };

/*
 * mxfp4_quantize -- x [out->rows x out->cols] (row stride ld_x elements) -> MXFP4 `out`.
 *   1. widen to fp32; for an E4M3 source v = fl(e4m3(b) * *src_scale), a NULL src_scale meaning 1.0;
 *   2. per 32-element block: b = max(E - 2, 0), E the exponent field of max |v| as fp32, i.e. the scale
 *      2^(floor(log2 max|v|) - 2) of the OCP conversion, not below 2^-127 (b = 0 for a zero block);
 *   3. per element: code = nearest E2M1 of v / 2^(b - 127) (exact division; ties to the even code,
 *      saturating at 6), sign bit = sign bit of v;
 *   4. a block that holds a NaN or an infinity gets b = 255 and zero codes (it reads back as NaN), and
 *      bit 0 is ORed into the optional *flags.
 * One launch, no workspace.  x_dtype any of nvfp4_dtype; src_scale only for NVFP4_E4M3.
 * src_scale and flags are device pointers.
 */
nvfp4_status mxfp4_quantize(const void *x, nvfp4_dtype x_dtype, int64_t ld_x, const float *src_scale,
                            const mxfp4_tensor *out, int32_t *flags, hipStream_t stream);

/*
 * mxfp4_dequantize -- MXFP4 `in` -> out [in->rows x in->cols] (row stride ld_out): e2m1 x 2^(b - 127),
 * exact in fp32 and in bf16 (above the largest finite value: infinity; b = 255: NaN).
 * out_dtype: NVFP4_F32 or NVFP4_BF16.  No workspace.
 */
nvfp4_status mxfp4_dequantize(const mxfp4_tensor *in, void *out, nvfp4_dtype out_dtype, int64_t ld_out,
                              hipStream_t stream);

/*
 * mxfp4_gemm -- C [M x N] (row stride ldc, fp32 or bf16) = A . W^T, with W an MXFP4 tensor [N x K] (a
 * PyTorch Linear weight, out-features x in-features) and A
 *   - a_q, an MXFP4 tensor [M x K] (W4A4), a_bf16 NULL; or
 *   - a_bf16 [M x K] bf16 (row stride lda; W4A16), a_q NULL.
 * Exactly one of the two must be given (NVFP4_ERR_ARG otherwise); lda is ignored for W4A4.  Products
 * are summed in fp32, subnormal numbers included, and rounded once to c_dtype (NVFP4_F32 or NVFP4_BF16).
 * W4A16 expands W on chip to bf16, which is exact below 2^128; a value of W beyond that (possible with scale
 * bytes 253 and 254 only) is an infinity there, as mxfp4_dequantize gives it.  A row of A with a NaN or an
 * infinity gives NaN or infinity in that row of C and nothing elsewhere; a NaN block of W gives NaN in its
 * column of C.
 * workspace (16-byte aligned, or NULL): with mxfp4_workspace_size(MXFP4_OP_GEMM_BF16 or _MX, M, N, K) bytes a
 * long K is split over workgroups where there are few output tiles (fp32 partial sums, added in slice
 * order); with less, or NULL, the product runs unsplit, in the tile shape that is cheapest then.  K <= 2^22,
 * and for M > 16 lda <= 2^22, M and N at most 2^31 - 2^11 (NVFP4_ERR_SHAPE).  K == 0 gives C = 0.
 */
nvfp4_status mxfp4_gemm(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                        void *c, nvfp4_dtype c_dtype, int64_t ldc, void *workspace, size_t workspace_bytes,
                        hipStream_t stream);

/*
 * mxfp4_moe -- a mixture-of-experts layer with MXFP4 experts, for up to MXFP4_MOE_MAX_TOKENS tokens:
 *   y[t] = sum over the experts e chosen for t of  p[t][e] . Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t]))
 * with silu(a) = a / (1 + exp(-a)), in two kernels.
 *   x       [tokens x H] bf16, row stride ld_x
 *   logits  [tokens x experts] fp32 or bf16 (logits_dtype), row stride ld_logits, element-aligned:
 *           the router's scores.  The top_k largest of a row are chosen, ties to the lowest expert.  A
 *           logit of -infinity masks its expert: such a row uses fewer than top_k experts, and none
 *           (y[t] = 0) when all are masked.  A row with a NaN or +infinity gives y[t] = NaN and no
 *           experts.
 *   p       the softmax over the chosen logits (renormalize = 1), or the chosen entries of the softmax
 *           over all of the row's logits (renormalize = 0)
 *   w_gate_up [experts * 2 I x H]: expert e's rows e * 2 I .. are I gate rows, then I up rows
 *   w_down    [experts * H x I]: expert e's rows start at e * H
 *   y       [tokens x H] fp32 or bf16 (y_dtype), row stride ld_y
 *   ids, weights  optional [tokens x top_k], dense: the chosen experts in descending order of logit and
 *           their p; -1 and 0 where a row has fewer
 * H and I are multiples of 32.  Weights are expanded to bf16 as in W4A16.  Sums are fp32, and the activations between the two products keep the bits of
 * fp32 (as three bf16 planes).  The result does not depend on the order of execution.
 * Errors: NVFP4_ERR_SHAPE for tokens > 64, experts > 512, top_k > 16, H or I above 2^22, or operands that
 * disagree; NVFP4_ERR_ARG for top_k < 1, top_k > experts or a bad renormalize; NVFP4_ERR_WORKSPACE for less than
 * mxfp4_workspace_size(MXFP4_OP_MOE, tokens * top_k, H, I) bytes (16-byte aligned).
 */
nvfp4_status mxfp4_moe(const void *x, int64_t tokens, int64_t ld_x, const void *logits, nvfp4_dtype logits_dtype,
                       int64_t ld_logits, int64_t experts, int top_k, int renormalize, const mxfp4_tensor *w_gate_up,
                       const mxfp4_tensor *w_down, void *y, nvfp4_dtype y_dtype, int64_t ld_y, int32_t *ids,
                       float *weights, void *workspace, size_t workspace_bytes, hipStream_t stream);

/* Largest arguments of the entry points below: (row, choice) pairs or grouped rows, and groups. */
enum { MXFP4_GROUP_MAX_ROWS = 1 << 24, MXFP4_MAX_GROUPS = MXFP4_MOE_MAX_EXPERTS };

/*
 * mxfp4_route -- the router of a mixture-of-experts layer, for any number of tokens: choices, weights and the
 * order of the rows that the products grouped by expert take.
 *   logits, renormalize   as for mxfp4_moe; logits [tokens x experts] fp32 or bf16, element-aligned rows
 *   ids      [tokens x top_k]: the chosen experts in descending order of logit, ties to the lowest expert;
 *            -1 where a row has fewer
 *   weights  [tokens x top_k]: their softmax weights; 0 where a row has fewer.  A row with a NaN or +infinity
 *            chooses no expert and has NaN for all its weights
 *   offsets  [experts + 1]: expert e has the positions offsets[e] .. offsets[e + 1] - 1
 *   rows     [tokens * top_k]: the token at each position, in the order of the tokens within an expert; -1 behind
 *            the last expert's
 *   places   [tokens x top_k]: the position of each choice, -1 where there is none
 * All outputs are required, dense and 4-byte aligned.  The result does not depend on the order of execution.
 * Errors: NVFP4_ERR_SHAPE for tokens * top_k > MXFP4_GROUP_MAX_ROWS, experts < 1 or > MXFP4_MAX_GROUPS, top_k >
 * MXFP4_MOE_MAX_TOP_K; NVFP4_ERR_ARG for top_k < 1, top_k > experts or a bad renormalize; NVFP4_ERR_WORKSPACE for less
 * than mxfp4_workspace_size(MXFP4_OP_ROUTE, tokens, top_k, experts) bytes (16-byte aligned; none for few tokens).
 */
nvfp4_status mxfp4_route(const void *logits, nvfp4_dtype logits_dtype, int64_t tokens, int64_t ld_logits, int64_t experts,
                         int top_k, int renormalize, int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                         int32_t *places, void *workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * mxfp4_group_rows -- the sort of mxfp4_route for choices that are given: ids [tokens x per_token] (dense) in 0 ..
 * groups - 1; any other value is no choice.  A token may name a group more than once.  places may be NULL.  Outputs,
 * limits (tokens * per_token, groups) and errors as for mxfp4_route; per_token >= 1 (NVFP4_ERR_ARG).
 */
nvfp4_status mxfp4_group_rows(const int32_t *ids, int64_t tokens, int per_token, int64_t groups, int32_t *offsets,
                              int32_t *rows, int32_t *places, void *workspace, size_t workspace_bytes,
                              hipStream_t stream);

/*
 * mxfp4_grouped_gemm -- products whose rows are grouped: for every group g and offsets[g] <= i < offsets[g + 1]
 *   C[i] = A[map[i]] . W[g]^T                                              (swiglu = 0), or
 *   C[i] = silu(A[map[i]] . Wg[g]^T) * (A[map[i]] . Wu[g]^T)               (swiglu = 1)
 * with silu(a) = a / (1 + exp(-a)).
 *   a_bf16 [a_rows x K] bf16 (row stride lda) or a_q, MXFP4 [a_rows x K]: exactly one (NVFP4_ERR_ARG otherwise)
 *   map      [rows] row of A of each row of C, or NULL for row i (then a_rows == rows).  A row outside 0 .. a_rows
 *            - 1 counts as zeros.
 *   offsets  [groups + 1] ascending.  They are read on the device; values outside 0 .. rows are cut off there.
 *   w        [groups * N x K] MXFP4, groups stacked by rows; with swiglu a group's rows are N / 2 gate rows, then N / 2
 *            up rows
 *   c        [rows x N] (swiglu: N / 2) fp32 or bf16, row stride ldc; or c_q, an MXFP4 tensor of that shape (swiglu
 *            only), as mxfp4_quantize makes it from the fp32 values.  Exactly one.
 * Sums and silu are fp32, rounded once to C.  A group may be empty; rows of C outside every group are left as they are.
 * W4A16 and W4A4 as for mxfp4_gemm.  No workspace.  K is not split over workgroups: a few rows in a few groups are slower than as
 * products of their own (mxfp4_gemm).
 * Errors: NVFP4_ERR_SHAPE for rows or a_rows > MXFP4_GROUP_MAX_ROWS, groups < 1 or > MXFP4_MAX_GROUPS, K == 0, K or
 * lda above 2^20, w->rows not a multiple of groups (with swiglu: of 2 groups), N above 2^24, with a map a_rows rows of A
 * of 2^31 bytes or more, with swiglu N / 2 rows of W of 2^30 bytes or more, more output tiles than one launch holds, or
 * operands that disagree.
 */
nvfp4_status mxfp4_grouped_gemm(const void *a_bf16, const mxfp4_tensor *a_q, int64_t a_rows, int64_t lda, const int32_t *map,
                                const int32_t *offsets, int64_t groups, int64_t rows, const mxfp4_tensor *w, int swiglu,
                                void *c, nvfp4_dtype c_dtype, int64_t ldc, const mxfp4_tensor *c_q, hipStream_t stream);

/*
 * mxfp4_combine -- y[t] = sum_j weights[t][j] . z[places[t][j]]: the rows that a token's choices gave back, weighted, in
 * the order of j.  z [z_rows x cols] fp32 or bf16 (row stride ld_z), places and weights [tokens x top_k] dense, y
 * [tokens x cols] fp32 or bf16 (row stride ld_y).  Sums are fp32, rounded once.  A place outside 0 .. z_rows - 1 counts
 * as a row of zeros, so a NaN weight still gives NaN.  Rows of z need the alignment of their element only.  top_k >= 1
 * (NVFP4_ERR_ARG), tokens * top_k <= MXFP4_GROUP_MAX_ROWS (NVFP4_ERR_SHAPE).
 */
nvfp4_status mxfp4_combine(const void *z, nvfp4_dtype z_dtype, int64_t z_rows, int64_t ld_z, const int32_t *places,
                           const float *weights, int64_t tokens, int top_k, int64_t cols, void *y, nvfp4_dtype y_dtype,
                           int64_t ld_y, hipStream_t stream);

/*
 * mxfp4_experts -- the mixture-of-experts layer of mxfp4_moe for any number of tokens: mxfp4_route, the gate and up
 * product with its silu, the down product and mxfp4_combine, in the order of those calls.  Arguments as for mxfp4_moe;
 * in between
 *   quantize_acts = 1  x and h = silu(g) * u are quantized to MXFP4 (W4A4), h from its fp32 value;
 *   quantize_acts = 0  x stays bf16 and h is rounded to bf16 (W4A16).
 * What an expert gives a token is rounded to y's type, then weighted and summed in fp32.  (mxfp4_moe keeps more bits
 * between its products and reads the weights of a few tokens' experts faster.)  ids, weights: optional, as mxfp4_route's.
 * A row with a NaN or +infinity among its logits gives y = NaN.
 * Errors as for mxfp4_moe, without its limit on tokens, and as for the calls named: tokens * top_k <=
 * MXFP4_GROUP_MAX_ROWS, H and I <= 2^20, ld_x <= 2^20, x below 2^31 bytes; NVFP4_ERR_WORKSPACE for less than
 * mxfp4_experts_workspace_size(...) bytes (16-byte aligned).
 */
nvfp4_status mxfp4_experts(const void *x, int64_t tokens, int64_t ld_x, const void *logits, nvfp4_dtype logits_dtype,
                           int64_t ld_logits, int64_t experts, int top_k, int renormalize, int quantize_acts,
                           const mxfp4_tensor *w_gate_up, const mxfp4_tensor *w_down, void *y, nvfp4_dtype y_dtype,
                           int64_t ld_y, int32_t *ids, float *weights, void *workspace, size_t workspace_bytes,
                           hipStream_t stream);
size_t mxfp4_experts_workspace_size(int64_t tokens, int64_t experts, int top_k, int64_t H, int64_t I, int quantize_acts,
                                    nvfp4_dtype y_dtype);

/* Largest arguments of mxfp4_gemm_adapters. */
enum { MXFP4_MAX_ADAPTERS = 1 << 16, MXFP4_MAX_RANK = 256 };

/*
 * mxfp4_gemm_adapters -- a projection that requests share, with low-rank adapters that are their own:
 *   C[m] = A[m] . W^T + s[i] (A[m] . V[i]^T) . U[i]^T,   i = index[m]
 *   a_bf16  [M x K] bf16, row stride lda: the activations of the branch, and of the product when a_q is NULL (W4A16)
 *   a_q     NULL, or the MXFP4 activations [M x K] of a W4A4 product
 *   w       [N x K] MXFP4
 *   index   [M]: the adapter of each row, in any order; outside 0 .. adapters - 1: none (the row is the product's)
 *   down    V [adapters x rank x K] bf16, up U [adapters x N x rank] bf16, dense; rank 8 .. MXFP4_MAX_RANK, a multiple of 8
 *           (an adapter of a lower rank is filled up with zeros)
 *   scales  [adapters] fp32, or NULL for 1
 *   c       [M x N] fp32 or bf16 (row stride ldc)
 * Sums are fp32 (A . V^T too, which passes on with fp32's 24 bits), and C is rounded once.  What an adapter holds reaches
 * the rows that name it and no others.  A NaN or infinity in V or U gives NaN or infinity in rows that name that adapter.
 * index, down, up and scales are read on the device.
 * Speed: with more than 64 rows and 2 to 511 adapters the rows are taken in the order of their adapters, so that a tile of C has
 * few.  With 512 adapters or more (however many the rows name), and where M * max(2 lda, K) reaches 2^31, they are taken as they
 * come, which costs as much where an adapter's rows lie side by side and several times as much where they are mixed: group them
 * before the call then, or pass the batch's own adapters alone.
 * workspace (16-byte aligned; none without adapters): with mxfp4_adapters_workspace_size(...) bytes a long K may be split as
 * in mxfp4_gemm; what that size is for K = 32 is needed in any case (NVFP4_ERR_WORKSPACE for less).  quantized_acts: whether
 * a_q is given.  M <= MXFP4_GROUP_MAX_ROWS, lda <= 2^21; else limits and errors as for mxfp4_gemm.
 */
nvfp4_status mxfp4_gemm_adapters(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                                 const int32_t *index, int64_t adapters, int64_t rank, const void *down, const void *up,
                                 const float *scales, void *c, nvfp4_dtype c_dtype, int64_t ldc, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream);
size_t mxfp4_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank, int quantized_acts);

/* Workspace bytes of an entry point (0 when none); see the selectors for the arguments.  Planned for
 * the current device (an MI355X's 256 CUs when none can be queried). */
size_t mxfp4_workspace_size(int op, int64_t m, int64_t n, int64_t k);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
