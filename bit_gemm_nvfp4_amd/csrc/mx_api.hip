// C ABI of the MXFP4 entry points (include/mxfp4.h): argument validation and dispatch.  Every entry
// point validates all of its arguments before enqueuing anything; none synchronizes, allocates or keeps
// a pointer.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mx.h"
#include "mx_adapters.h"
#include "mx_plan.h"
#include "mxfp4.h"

#include <algorithm>
#include <initializer_list>

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

// Products grouped by rows: rows of A and W short enough for the 256 that share a buffer to stay within 2^29 bytes.
constexpr int64_t kMaxGroupK = (int64_t)1 << 20, kMaxGroupN = (int64_t)1 << 24;
constexpr int64_t kMaxAdapterLd = (int64_t)1 << 21;  // (2^30 bytes)

// Whether the tiles of a grouped product fit one launch.
bool grouped_fits(int64_t rows, int64_t groups, int64_t N, int64_t K, bool a_mx, int cus) {
    return rows == 0 || N == 0 || plan_grouped(rows, groups, N, K, a_mx, cus) >= 0;
}

bool pairs_fit(int64_t rows, int64_t per) {
    return rows >= 0 && per >= 0 && (per == 0 || rows <= MXFP4_GROUP_MAX_ROWS / per);
}

nvfp4_status check_words(const void *p, bool needed) {
    if (!p) return needed ? NVFP4_ERR_NULL : NVFP4_OK;
    return aligned(p, 4) ? NVFP4_OK : NVFP4_ERR_ALIGN;
}

// The first of these that is not NVFP4_OK.
nvfp4_status first_of(std::initializer_list<nvfp4_status> all) {
    for (nvfp4_status s : all)
        if (s != NVFP4_OK) return s;
    return NVFP4_OK;
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// The workspace of mxfp4_gemm_adapters: T (fp32, or three bf16 planes); the branch's sums where it has them; where the rows
// are sorted by adapter their order, the groups' offsets and the sort's own workspace; then the product's.
struct AdaptersWs {
    size_t sums, order, offsets, sort, product;
    bool few, sorted, summed;
};
AdaptersWs adapters_ws(int64_t M, int64_t N, int64_t rank, int64_t adapters) {
    AdaptersWs w{};
    w.few = M <= kAdapterElementRows;
    w.summed = w.few && M > 16;  // (with fewer the product forms them)
    w.sorted = !w.few && adapters > 1 && adapters < MXFP4_MAX_GROUPS;
    w.sums = align256((size_t)M * rank * (w.few ? 4 : 2 * kAdapterPlanes));
    w.order = w.sums + (w.summed ? align256((size_t)M * N * 4) : 0);
    w.offsets = w.order + (w.sorted ? align256((size_t)M * 4) : 0);
    w.sort = w.offsets + (w.sorted ? align256((size_t)(adapters + 2) * 4) : 0);
    w.product = w.sort + (w.sorted ? align256(mx_sort_ws_bytes(M, adapters + 1)) : 0);
    return w;
}

bool rank_fits(int64_t rank) { return rank >= 8 && rank <= MXFP4_MAX_RANK && rank % 8 == 0; }

// Parts of the workspace of mxfp4_experts, each 256-byte aligned.
struct ExpertsWs {
    size_t ids, weights, offsets, rows, places, sort, xq_codes, xq_scales, h, h_scales, z, total;
    size_t sort_bytes;
};
ExpertsWs experts_ws(int64_t tokens, int64_t experts, int top_k, int64_t H, int64_t I, bool quantize, int yeb) {
    ExpertsWs w{};
    const size_t pairs = (size_t)(tokens * top_k);
    size_t at = 0;
    auto part = [&](size_t bytes) {
        const size_t here = at;
        at += align256(bytes);
        return here;
    };
    w.sort_bytes = mx_route_ws_bytes(tokens, top_k, experts);
    w.ids = part(pairs * 4);
    w.weights = part(pairs * 4);
    w.offsets = part((size_t)(experts + 1) * 4);
    w.rows = part(pairs * 4);
    w.places = part(pairs * 4);
    w.sort = part(w.sort_bytes);
    w.xq_codes = part(quantize ? (size_t)tokens * (H / 2) : 0);
    w.xq_scales = part(quantize ? (size_t)tokens * (H / kMxBlock) : 0);
    w.h = part(pairs * (quantize ? I / 2 : I * 2));
    w.h_scales = part(quantize ? pairs * (I / kMxBlock) : 0);
    w.z = part(pairs * (size_t)H * yeb);
    w.total = tokens > 0 ? at : 0;
    return w;
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
    case MXFP4_OP_ROUTE: return pairs_fit(m, n) && k <= MXFP4_MAX_GROUPS ? mx_route_ws_bytes(m, n, k) : 0;
    case MXFP4_OP_GROUP_ROWS: return pairs_fit(m, n) && k <= MXFP4_MAX_GROUPS ? mx_sort_ws_bytes(m * n, k) : 0;
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

nvfp4_status mxfp4_route(const void *logits, nvfp4_dtype logits_dtype, int64_t tokens, int64_t ld_logits, int64_t experts,
                         int top_k, int renormalize, int32_t *ids, float *weights, int32_t *offsets, int32_t *rows,
                         int32_t *places, void *workspace, size_t workspace_bytes, hipStream_t stream) {
    if (logits_dtype != NVFP4_F32 && logits_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    if (tokens < 0 || experts < 1 || experts > MXFP4_MAX_GROUPS || top_k > MXFP4_MOE_MAX_TOP_K) return NVFP4_ERR_SHAPE;
    if (top_k < 1 || top_k > experts || (renormalize != 0 && renormalize != 1)) return NVFP4_ERR_ARG;
    if (!pairs_fit(tokens, top_k)) return NVFP4_ERR_SHAPE;
    const int leb = elem_bytes(logits_dtype);
    const bool any = tokens > 0;
    const nvfp4_status st = first_of({check_rows(logits, tokens, experts, ld_logits, leb, leb), check_words(ids, any),
                                      check_words(weights, any), check_words(offsets, true), check_words(rows, any),
                                      check_words(places, any)});
    if (st != NVFP4_OK) return st;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    if (mx_route_ws_bytes(tokens, top_k, experts) > (workspace ? workspace_bytes : 0)) return NVFP4_ERR_WORKSPACE;
    if (current_device_cus() == 0) return NVFP4_ERR_DEVICE;
    const MxRouteArgs a{logits,      logits_dtype == NVFP4_BF16, tokens, ld_logits, experts, top_k,
                        renormalize, ids,                        weights, offsets,  rows,    places};
    return launched(launch_mx_route(a, workspace, stream));
}

nvfp4_status mxfp4_group_rows(const int32_t *ids, int64_t tokens, int per_token, int64_t groups, int32_t *offsets,
                              int32_t *rows, int32_t *places, void *workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    if (tokens < 0 || groups < 1 || groups > MXFP4_MAX_GROUPS) return NVFP4_ERR_SHAPE;
    if (per_token < 1) return NVFP4_ERR_ARG;
    if (!pairs_fit(tokens, per_token)) return NVFP4_ERR_SHAPE;
    const nvfp4_status st = first_of({check_words(ids, tokens > 0), check_words(offsets, true),
                                      check_words(rows, tokens > 0), check_words(places, false)});
    if (st != NVFP4_OK) return st;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    if (mx_sort_ws_bytes(tokens * per_token, groups) > (workspace ? workspace_bytes : 0)) return NVFP4_ERR_WORKSPACE;
    if (current_device_cus() == 0) return NVFP4_ERR_DEVICE;
    return launched(launch_mx_sort(ids, tokens, per_token, groups, offsets, rows, places, false, workspace, stream));
}

nvfp4_status mxfp4_grouped_gemm(const void *a_bf16, const mxfp4_tensor *a_q, int64_t a_rows, int64_t lda, const int32_t *map,
                                const int32_t *offsets, int64_t groups, int64_t rows, const mxfp4_tensor *w, int swiglu,
                                void *c, nvfp4_dtype c_dtype, int64_t ldc, const mxfp4_tensor *c_q, hipStream_t stream) {
    nvfp4_status st = check_mx(w);
    if (st != NVFP4_OK) return st;
    const int64_t K = w->cols;
    if (rows < 0 || rows > MXFP4_GROUP_MAX_ROWS || a_rows < 0 || a_rows > MXFP4_GROUP_MAX_ROWS || groups < 1 ||
        groups > MXFP4_MAX_GROUPS || K == 0 || K > kMaxGroupK)
        return NVFP4_ERR_SHAPE;
    if ((swiglu != 0 && swiglu != 1) || (a_bf16 && a_q) || (c && c_q) || (c_q && !swiglu)) return NVFP4_ERR_ARG;
    const int64_t parts = swiglu ? 2 * groups : groups;
    if (w->rows % parts != 0 || w->rows / groups > kMaxGroupN) return NVFP4_ERR_SHAPE;
    const int64_t cols = w->rows / parts;
    if (swiglu && cols * (K / 2) >= (int64_t)1 << 30) return NVFP4_ERR_SHAPE;
    if (!map && a_rows != rows) return NVFP4_ERR_SHAPE;
    if (!a_bf16 && !a_q && a_rows > 0) return NVFP4_ERR_ARG;
    if (a_q) {
        st = check_mx(a_q);
        if (st != NVFP4_OK) return st;
        if (a_q->rows != a_rows || a_q->cols != K) return NVFP4_ERR_SHAPE;
    } else {
        st = check_rows(a_bf16, a_rows, K, lda, 2, 16);
        if (st != NVFP4_OK) return st;
        if (lda > kMaxGroupK) return NVFP4_ERR_SHAPE;
    }
    if (map && a_rows * (a_q ? K / 2 : lda * 2) >= (int64_t)1 << 31) return NVFP4_ERR_SHAPE;
    if (c_q) {
        st = check_mx(c_q);
        if (st != NVFP4_OK) return st;
        if (c_q->rows != rows || c_q->cols != cols) return NVFP4_ERR_SHAPE;
    } else {
        if (c_dtype != NVFP4_F32 && c_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
        const int eb = elem_bytes(c_dtype);
        st = check_rows(c, rows, cols, ldc, eb, eb);
        if (st != NVFP4_OK) return st;
    }
    st = first_of({check_words(map, false), check_words(offsets, true)});
    if (st != NVFP4_OK) return st;
    const int cus = current_device_cus();
    if (cus == 0) return NVFP4_ERR_DEVICE;
    if (!grouped_fits(rows, groups, w->rows / groups, K, a_q != nullptr, cus)) return NVFP4_ERR_SHAPE;
    if (rows == 0 || cols == 0) return NVFP4_OK;
    const MxGroupedArgs a{a_bf16, a_q, a_rows, lda, map, offsets, groups, rows, w, swiglu == 1, c, c_dtype, ldc, c_q};
    return launched(launch_mx_grouped(a, cus, stream));
}

nvfp4_status mxfp4_combine(const void *z, nvfp4_dtype z_dtype, int64_t z_rows, int64_t ld_z, const int32_t *places,
                           const float *weights, int64_t tokens, int top_k, int64_t cols, void *y, nvfp4_dtype y_dtype,
                           int64_t ld_y, hipStream_t stream) {
    if ((z_dtype != NVFP4_F32 && z_dtype != NVFP4_BF16) || (y_dtype != NVFP4_F32 && y_dtype != NVFP4_BF16))
        return NVFP4_ERR_DTYPE;
    if (tokens < 0 || z_rows < 0 || z_rows > kMaxDim || cols > kMaxDim) return NVFP4_ERR_SHAPE;
    if (top_k < 1) return NVFP4_ERR_ARG;
    if (!pairs_fit(tokens, top_k)) return NVFP4_ERR_SHAPE;
    const int zeb = elem_bytes(z_dtype), yeb = elem_bytes(y_dtype);
    const nvfp4_status st =
        first_of({check_rows(z, z_rows, cols, ld_z, zeb, zeb), check_rows(y, tokens, cols, ld_y, yeb, yeb),
                  check_words(places, tokens > 0), check_words(weights, tokens > 0)});
    if (st != NVFP4_OK) return st;
    if (current_device_cus() == 0) return NVFP4_ERR_DEVICE;
    if (tokens == 0 || cols == 0) return NVFP4_OK;
    return launched(launch_mx_combine(z, z_dtype, z_rows, ld_z, places, weights, tokens, top_k, cols, y, y_dtype, ld_y, stream));
}

size_t mxfp4_experts_workspace_size(int64_t tokens, int64_t experts, int top_k, int64_t H, int64_t I, int quantize_acts,
                                    nvfp4_dtype y_dtype) {
    if (tokens < 0 || top_k < 1 || !pairs_fit(tokens, top_k) || experts < 1 || experts > MXFP4_MAX_GROUPS || H < 0 ||
        H > kMaxGroupK || I < 0 || I > kMaxGroupK || (y_dtype != NVFP4_F32 && y_dtype != NVFP4_BF16))
        return 0;
    return experts_ws(tokens, experts, top_k, H, I, quantize_acts != 0, elem_bytes(y_dtype)).total;
}

nvfp4_status mxfp4_experts(const void *x, int64_t tokens, int64_t ld_x, const void *logits, nvfp4_dtype logits_dtype,
                           int64_t ld_logits, int64_t experts, int top_k, int renormalize, int quantize_acts,
                           const mxfp4_tensor *w_gate_up, const mxfp4_tensor *w_down, void *y, nvfp4_dtype y_dtype,
                           int64_t ld_y, int32_t *ids, float *weights, void *workspace, size_t workspace_bytes,
                           hipStream_t stream) {
    if (logits_dtype != NVFP4_F32 && logits_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    if (y_dtype != NVFP4_F32 && y_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    nvfp4_status st = first_of({check_mx(w_gate_up), check_mx(w_down)});
    if (st != NVFP4_OK) return st;
    if (tokens < 0 || experts < 1 || experts > MXFP4_MAX_GROUPS || top_k > MXFP4_MOE_MAX_TOP_K) return NVFP4_ERR_SHAPE;
    if (top_k < 1 || top_k > experts || (renormalize != 0 && renormalize != 1) ||
        (quantize_acts != 0 && quantize_acts != 1))
        return NVFP4_ERR_ARG;
    const int64_t H = w_gate_up->cols, I = w_down->cols;
    if (H == 0 || I == 0 || H > kMaxGroupK || I > kMaxGroupK || w_gate_up->rows != experts * 2 * I ||
        w_down->rows != experts * H || !pairs_fit(tokens, top_k) || I * (H / 2) >= (int64_t)1 << 30)
        return NVFP4_ERR_SHAPE;
    const int leb = elem_bytes(logits_dtype), yeb = elem_bytes(y_dtype);
    st = first_of({check_rows(x, tokens, H, ld_x, 2, 16), check_rows(logits, tokens, experts, ld_logits, leb, leb),
                   check_rows(y, tokens, H, ld_y, yeb, yeb)});
    if (st != NVFP4_OK) return st;
    if (ld_x > kMaxGroupK || tokens * ld_x * 2 >= (int64_t)1 << 31) return NVFP4_ERR_SHAPE;
    if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    const ExpertsWs at = experts_ws(tokens, experts, top_k, H, I, quantize_acts == 1, yeb);
    if (at.total > (workspace ? workspace_bytes : 0)) return NVFP4_ERR_WORKSPACE;
    const int cus = current_device_cus();
    if (cus == 0) return NVFP4_ERR_DEVICE;
    if (!grouped_fits(tokens * top_k, experts, 2 * I, H, quantize_acts == 1, cus) ||
        !grouped_fits(tokens * top_k, experts, H, I, quantize_acts == 1, cus))
        return NVFP4_ERR_SHAPE;
    if (tokens == 0) return NVFP4_OK;

    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    auto words = [&](size_t part) { return reinterpret_cast<int32_t *>(ws + part); };
    const int64_t pairs = tokens * top_k;
    int32_t *const chosen = ids ? ids : words(at.ids), *const offsets = words(at.offsets);
    float *const wts = weights ? weights : reinterpret_cast<float *>(ws + at.weights);
    const MxRouteArgs route{logits,      logits_dtype == NVFP4_BF16, tokens, ld_logits, experts,        top_k,
                            renormalize, chosen,                     wts,    offsets,   words(at.rows), words(at.places)};
    hipError_t e = launch_mx_route(route, ws + at.sort, stream);
    if (e != hipSuccess) return launched(e);
    const mxfp4_tensor xq{ws + at.xq_codes, ws + at.xq_scales, tokens, H}, hq{ws + at.h, ws + at.h_scales, pairs, I};
    if (quantize_acts) {
        e = launch_mx_quantize(x, NVFP4_BF16, ld_x, nullptr, &xq, nullptr, stream);
        if (e != hipSuccess) return launched(e);
    }
    MxGroupedArgs up{}, down{};
    up.a_rows = tokens;
    up.lda = ld_x;
    up.map = words(at.rows);
    up.offsets = down.offsets = offsets;
    up.groups = down.groups = experts;
    up.rows = down.rows = down.a_rows = pairs;
    up.w = w_gate_up;
    up.swiglu = true;
    down.lda = up.ldc = I;
    down.w = w_down;
    down.c = ws + at.z;
    down.c_dtype = y_dtype;
    down.ldc = H;
    up.c_dtype = NVFP4_BF16;
    if (quantize_acts) {
        up.a_q = &xq;
        up.c_q = down.a_q = &hq;
    } else {
        up.a_bf16 = x;
        up.c = ws + at.h;
        down.a_bf16 = ws + at.h;
    }
    e = launch_mx_grouped(up, cus, stream);
    if (e != hipSuccess) return launched(e);
    e = launch_mx_grouped(down, cus, stream);
    if (e != hipSuccess) return launched(e);
    return launched(launch_mx_combine(ws + at.z, y_dtype, pairs, H, words(at.places), wts, tokens, top_k, H, y, y_dtype, ld_y, stream));
}

size_t mxfp4_adapters_workspace_size(int64_t M, int64_t N, int64_t K, int64_t adapters, int64_t rank, int quantized_acts) {
    if (M <= 0 || M > MXFP4_GROUP_MAX_ROWS || N <= 0 || N > kMaxDim || K <= 0 || K > kMaxDim || adapters < 0 ||
        adapters > MXFP4_MAX_ADAPTERS || !rank_fits(rank))
        return 0;
    const int cus = current_device_cus();
    const AdaptersWs at = adapters_ws(M, N, rank, adapters);
    return (adapters > 0 ? at.product : 0) + mx_gemm_ws_bytes(M, N, K, quantized_acts != 0, cus > 0 ? cus : 256,
                                                              adapters > 0 && at.summed ? kFirstLowShape : 0);
}

nvfp4_status mxfp4_gemm_adapters(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                                 const int32_t *index, int64_t adapters, int64_t rank, const void *down, const void *up,
                                 const float *scales, void *c, nvfp4_dtype c_dtype, int64_t ldc, void *workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    nvfp4_status st = check_mx(w);
    if (st != NVFP4_OK) return st;
    const int64_t N = w->rows, K = w->cols;
    if (c_dtype != NVFP4_F32 && c_dtype != NVFP4_BF16) return NVFP4_ERR_DTYPE;
    if (M < 0 || M > MXFP4_GROUP_MAX_ROWS || K > kMaxK || (M > 16 && N > kMaxTileDim) || adapters < 0 ||
        adapters > MXFP4_MAX_ADAPTERS || !rank_fits(rank))
        return NVFP4_ERR_SHAPE;
    st = check_rows(a_bf16, M, K, lda, 2, 16);
    if (st != NVFP4_OK) return st;
    if (lda > kMaxAdapterLd) return NVFP4_ERR_SHAPE;
    if (a_q) {
        st = check_mx(a_q);
        if (st != NVFP4_OK) return st;
        if (a_q->rows != M || a_q->cols != K) return NVFP4_ERR_SHAPE;
    }
    const int eb = elem_bytes(c_dtype);
    st = first_of({check_rows(down, adapters * rank, K, K, 2, 16), check_rows(up, adapters * N, rank, rank, 2, 16),
                   check_rows(c, M, N, ldc, eb, eb), check_words(index, M > 0), check_words(scales, false)});
    if (st != NVFP4_OK) return st;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
    const size_t have = workspace ? workspace_bytes : 0;
    const bool branch = M > 0 && N > 0 && K > 0 && adapters > 0;
    const AdaptersWs at = adapters_ws(M, N, rank, adapters);
    if (branch && have < at.product) return NVFP4_ERR_WORKSPACE;
    const int cus = current_device_cus();
    if (cus == 0) return NVFP4_ERR_DEVICE;
    if (M == 0 || N == 0) return NVFP4_OK;
    uint8_t *const ws = reinterpret_cast<uint8_t *>(workspace);
    if (!branch) return launched(launch_mx_gemm(a_q ? nullptr : a_bf16, a_q, M, lda, w, c, c_dtype, ldc, ws, have, cus, stream));
    float *const t = at.few ? reinterpret_cast<float *>(ws) : nullptr, *const sums = at.summed ? reinterpret_cast<float *>(ws + at.sums) : nullptr;
    __bf16 *const t_planes = t ? nullptr : reinterpret_cast<__bf16 *>(ws);
    // rows in another order are picked from one buffer of all of A
    int32_t *const order = at.sorted && M * std::max(lda * 2, K) < ((int64_t)1 << 31) ? reinterpret_cast<int32_t *>(ws + at.order) : nullptr;
    hipError_t e = hipSuccess;
    if (order)
        e = launch_mx_sort(index, M, 1, adapters + 1, reinterpret_cast<int32_t *>(ws + at.offsets), order, nullptr, true, ws + at.sort, stream);
    if (e != hipSuccess) return launched(e);
    e = launch_adapter_down(AdapterDownArgs{a_bf16, M, lda, K, down, scales, index, order, (int)adapters, (int)rank, t, t_planes}, cus, stream);
    if (e != hipSuccess) return launched(e);
    const Adapters ad{t, t_planes, sums, reinterpret_cast<const __bf16 *>(up), index, order, (int)adapters, (int)rank};
    if (sums) e = launch_adapter_sums(ad, M, N, sums, stream);
    if (e != hipSuccess) return launched(e);
    return launched(launch_mx_gemm(a_q ? nullptr : a_bf16, a_q, M, lda, w, c, c_dtype, ldc, ws + at.product, have - at.product, cus,
                                   stream, &ad));
}

}  // extern "C"
