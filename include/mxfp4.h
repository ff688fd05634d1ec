/*
 * mxfp4.h -- MXFP4 entry points of libnvfp4.so: block quantization with power-of-two scales, its
 * expansion, the product with MXFP4 weights and a mixture-of-experts layer for a few tokens, as
 * hand-written HIP kernels for AMD Instinct MI355X (gfx950).
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
    MXFP4_OP_MOE = 2        /* mxfp4_moe: (tokens * top_k, H, I)                               */
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

/* Workspace bytes of an entry point (0 when none); see the selectors for the arguments.  Planned for
 * the current device (an MI355X's 256 CUs when none can be queried). */
size_t mxfp4_workspace_size(int op, int64_t m, int64_t n, int64_t k);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */
