// C ABI of the MXFP4 entry points (include/mxfp4.h): argument validation and dispatch.  Every entry
// point validates all of its arguments before enqueuing anything; none synchronizes, allocates or keeps
// a pointer.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mx.h"
#include "mxfp4.h"

using namespace nvfp4;

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int elem_bytes(nvfp4_dtype dt) {
    switch (dt) {
    case NVFP4_F32: return 4;
    case NVFP4_BF16:
    case NVFP4_F16: return 2;
    case NVFP4_E4M3: return 1;
    default: return 0;
    }
}

// Sizes the kernels index with: rows and columns below 2^31, rows short enough for those that share a buffer to stay
// within 2^29 bytes (64 rows of A, 256 rows of W), the limits themselves included.
constexpr int64_t kMaxDim = 0x7FFFFFFF, kMaxK = (int64_t)1 << 22, kMaxTileLd = (int64_t)1 << 22;
// Rows whose tiles fit one launch in the largest tile shape.
constexpr int64_t kMaxTileDim = ((int64_t)1 << 31) - (1 << 11);

nvfp4_status check_mx(const mxfp4_tensor *t) {
    if (!t) return NVFP4_ERR_NULL;
    if (t->rows < 0 || t->cols < 0 || t->cols % kMxBlock != 0 || t->rows > kMaxDim || t->cols > kMaxDim)
        return NVFP4_ERR_SHAPE;
    if (t->rows == 0 || t->cols == 0) return NVFP4_OK;
    if (!t->codes || !t->scales) return NVFP4_ERR_NULL;
    return aligned(t->codes, 16) && aligned(t->scales, 16) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// A row-major matrix whose pointer and row starts are `align`-byte aligned; NULL only without elements.
nvfp4_status check_rows(const void *p, int64_t rows, int64_t cols, int64_t ld, int eb, int align) {
    if (rows < 0 || cols < 0 || ld < cols || ld > kMaxDim) return NVFP4_ERR_SHAPE;
    if (rows == 0 || cols == 0) return NVFP4_OK;
    if (!p) return NVFP4_ERR_NULL;
    if (!aligned(p, align) || (rows > 1 && (ld * eb) % align != 0)) return NVFP4_ERR_ALIGN;
    return NVFP4_OK;
}

nvfp4_status launched(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_LAUNCH; }

}  // namespace

extern "C" {

size_t mxfp4_workspace_size(int op, int64_t m, int64_t n, int64_t k) {
    if (m < 0 || n < 0 || k < 0 || m > kMaxDim || n > kMaxDim || k > kMaxDim) return 0;
    const int cus = current_device_cus();
    switch (op) {
    case MXFP4_OP_GEMM_BF16: return mx_gemm_ws_bytes(m, n, k, false, cus > 0 ? cus : 256);
    case MXFP4_OP_GEMM_MX: return mx_gemm_ws_bytes(m, n, k, true, cus > 0 ? cus : 256);
    case MXFP4_OP_MOE:
        if (m > MXFP4_MOE_MAX_TOKENS * MXFP4_MOE_MAX_TOP_K) return 0;
        return mx_moe_ws_bytes(m, n, k);
    default: return 0;
    }
}

nvfp4_status mxfp4_quantize(const void *x, nvfp4_dtype x_dtype, int64_t ld_x, const float *src_scale,
                            const mxfp4_tensor *out, int32_t *flags, hipStream_t stream) {
    const int eb = elem_bytes(x_dtype);
    if (eb == 0) return NVFP4_ERR_DTYPE;
    nvfp4_status st = check_mx(out);
    if (st != NVFP4_OK) return st;
    st = check_rows(x, out->rows, out->cols, ld_x, eb, 16);
    if (st != NVFP4_OK) return st;
    if (src_scale && x_dtype != NVFP4_E4M3) return NVFP4_ERR_ARG;
    if (!aligned(src_scale, 4) || !aligned(flags, 4)) return NVFP4_ERR_ALIGN;
    if (current_device_cus() == 0) return NVFP4_ERR_DEVICE;
    if (out->rows == 0 || out->cols == 0) return NVFP4_OK;
    return launched(launch_mx_quantize(x, x_dtype, ld_x, src_scale, out, flags, stream));
}

nvfp4_status mxfp4_dequantize(const mxfp4_tensor *in, void *out, nvfp4_dtype out_dtype, int64_t ld_out,
                              hipStream_t stream) {
    nvfp4_status st = check_mx(in);
    if (st != NVFP4_OK) return st;
    if (out_dtype != NVFP4_F32 && out_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    st = check_rows(out, in->rows, in->cols, ld_out, elem_bytes(out_dtype), 16);
    if (st != NVFP4_OK) return st;
    if (current_device_cus() == 0) return NVFP4_ERR_DEVICE;
    if (in->rows == 0 || in->cols == 0) return NVFP4_OK;
    return launched(launch_mx_dequantize(in, out, out_dtype, ld_out, stream));
}

nvfp4_status mxfp4_gemm(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                        void *c, nvfp4_dtype c_dtype, int64_t ldc, void *workspace, size_t workspace_bytes,
                        hipStream_t stream) {
    nvfp4_status st = check_mx(w);
    if (st != NVFP4_OK) return st;
    const int64_t N = w->rows, K = w->cols;
    if (c_dtype != NVFP4_F32 && c_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    if (M < 0 || M > kMaxDim || K > kMaxK) return NVFP4_ERR_SHAPE;
    if (M > 16 && (M > kMaxTileDim || N > kMaxTileDim)) return NVFP4_ERR_SHAPE;
    // rows of A without elements need no pointer
    if (a_bf16 && a_q) return NVFP4_ERR_ARG;
    if (!a_bf16 && !a_q && M > 0 && K > 0) return NVFP4_ERR_ARG;
    if (a_q) {
        st = check_mx(a_q);
        if (st != NVFP4_OK) return st;
        if (a_q->rows != M || a_q->cols != K) return NVFP4_ERR_SHAPE;
    } else {
        st = check_rows(a_bf16, M, K, lda, 2, 16);
        if (st != NVFP4_OK) return st;
        if (M > 16 && lda > kMaxTileLd) return NVFP4_ERR_SHAPE;
    }
    const int eb = elem_bytes(c_dtype);
    st = check_rows(c, M, N, ldc, eb, eb);
    if (st != NVFP4_OK) return st;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    const int cus = current_device_cus();
    if (cus == 0) return NVFP4_ERR_DEVICE;
    if (M == 0 || N == 0) return NVFP4_OK;
    return launched(launch_mx_gemm(a_bf16, a_q, M, lda, w, c, c_dtype, ldc, workspace, workspace_bytes, cus, stream));
}

nvfp4_status mxfp4_moe(const void *x, int64_t tokens, int64_t ld_x, const void *logits, nvfp4_dtype logits_dtype,
                       int64_t ld_logits, int64_t experts, int top_k, int renormalize, const mxfp4_tensor *w_gate_up,
                       const mxfp4_tensor *w_down, void *y, nvfp4_dtype y_dtype, int64_t ld_y, int32_t *ids,
                       float *weights, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (logits_dtype != NVFP4_F32 && logits_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    if (y_dtype != NVFP4_F32 && y_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    nvfp4_status st = check_mx(w_gate_up);
    if (st != NVFP4_OK) return st;
    st = check_mx(w_down);
    if (st != NVFP4_OK) return st;
    if (tokens < 0 || tokens > MXFP4_MOE_MAX_TOKENS || experts < 1 || experts > MXFP4_MOE_MAX_EXPERTS ||
        top_k > MXFP4_MOE_MAX_TOP_K)
        return NVFP4_ERR_SHAPE;
    if (top_k < 1 || top_k > experts || (renormalize != 0 && renormalize != 1)) return NVFP4_ERR_ARG;
    const int64_t H = w_gate_up->cols, I = w_down->cols;
    if (H == 0 || I == 0 || H > kMaxK || I > kMaxK || w_gate_up->rows != experts * 2 * I ||
        w_down->rows != experts * H)
        return NVFP4_ERR_SHAPE;
    st = check_rows(x, tokens, H, ld_x, 2, 16);
    if (st != NVFP4_OK) return st;
    const int leb = elem_bytes(logits_dtype), yeb = elem_bytes(y_dtype);
    st = check_rows(logits, tokens, experts, ld_logits, leb, leb);
    if (st != NVFP4_OK) return st;
    st = check_rows(y, tokens, H, ld_y, yeb, yeb);
    if (st != NVFP4_OK) return st;
    if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    if (tokens > 0 && (!workspace || workspace_bytes < mx_moe_ws_bytes(tokens * top_k, H, I))) return NVFP4_ERR_WORKSPACE;
    const int cus = current_device_cus();
    if (cus == 0) return NVFP4_ERR_DEVICE;
    if (tokens == 0) return NVFP4_OK;
    const MoeArgs a{x,     tokens,      ld_x,   logits, logits_dtype == NVFP4_BF16, ld_logits, experts, top_k,
                    renormalize, w_gate_up, w_down, y,      y_dtype == NVFP4_BF16,      ld_y,      ids,     weights};
    return launched(launch_mx_moe(a, workspace, cus, stream));
}

}  // extern "C"
