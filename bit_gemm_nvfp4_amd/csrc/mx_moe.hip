// Mixture-of-experts layer with MXFP4 experts for a few tokens (gfx950), in two kernels:
//   y[t] = sum_e p[t][e] . Wd[e] (silu(Wg[e] x[t]) * (Wu[e] x[t])), e over the top-k of logits[t].
//
// Bound by streaming the chosen experts' weights (17/32 byte per element) once from HBM; everything else
// is small.  Weights go from memory to registers in the matrix instructions' operand layout (MxGroup),
// are expanded exactly to bf16 (half an instruction per element) and multiply 16 tokens at a time with
// v_mfma_f32_16x16x32_bf16.
//
// Routing needs no kernel of its own: an expert's rank in a row is the number of entries ahead of it
// (larger, or equal with a lower index), so a workgroup of the first kernel finds which tokens chose its
// expert by counting, and one further workgroup per token writes that token's choices and softmax sum.
//   k_moe_up:   workgroup (slot, 16 intermediate rows): gate and up products of the slot's expert for
//               the tokens that chose it, h = silu(g) u exp(logit - row max), stored as two bf16 planes
//               (2^-17 of its value) per (token, choice).  With tokens * top_k < experts a slot is a
//               (token, choice) pair, and the workgroups of a pair whose expert an earlier token chose
//               leave; otherwise a slot is an expert.
//   k_moe_down: workgroup (16 rows of Wd): all chosen experts, (expert, 512-column group) items dealt to
//               the waves; the accumulators run over experts, since h carries the softmax weight; the
//               row's softmax sum divides at the end.  No atomics: sums are joined in wave order.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mx.h"

namespace nvfp4 {

namespace {

constexpr int kMaxT = MXFP4_MOE_MAX_TOKENS, kMaxE = MXFP4_MOE_MAX_EXPERTS, kMaxK = MXFP4_MOE_MAX_TOP_K;
constexpr int kUpWaves = 4, kDownWaves = 8;

struct MoeDev {
    const __bf16 *x;
    const void *logits;
    int64_t ld_x, ld_logits;
    const uint8_t *gu_codes, *gu_scales, *dn_codes, *dn_scales;
    int64_t H, I;
    void *y;
    int64_t ld_y;
    int32_t *ids;       // user's, may be null
    float *weights;     // user's, may be null
    int32_t *ws_ids;    // [T][k]
    float *ws_den;      // [T] softmax sum; NaN for a row with NaN or +inf
    __bf16 *h_hi, *h_lo;  // [T * k][I]
    int T, E, k, renorm, slots, pair_slots, tiles;
};

template <bool BF16>
__device__ __forceinline__ float load_logit(const MoeDev &a, int t, int e) {
    if constexpr (BF16) return (float)reinterpret_cast<const __bf16 *>(a.logits)[(int64_t)t * a.ld_logits + e];
    else return reinterpret_cast<const float *>(a.logits)[(int64_t)t * a.ld_logits + e];
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + expf(-g)); }

__device__ __forceinline__ bool is_bad(float v) { return !(v < __builtin_inff()); }  // NaN or +inf

__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    return v;
}

// Rank of expert e in row t (one wave, every lane gets the result), the row maximum, and whether the row
// holds a NaN or +inf.
template <bool BF16>
__device__ __forceinline__ int wave_rank(const MoeDev &a, int t, int e, int lane, float &le, float &top, bool &bad) {
    le = load_logit<BF16>(a, t, e);
    int n = 0;
    bool b = false;
    float m = -__builtin_inff();
    for (int j = lane; j < a.E; j += 64) {
        const float v = load_logit<BF16>(a, t, j);
        b = b || is_bad(v);
        m = fmaxf(m, v);
        n += (v > le || (v == le && j < e)) ? 1 : 0;
    }
    top = wave_max_f32(m);
    bad = __any(b);
    return (int)wave_sum_u32((uint32_t)n);
}

// One token's choices and softmax sum (a whole workgroup of 256).
template <bool BF16>
__device__ void route_token(const MoeDev &a, int t, float *row, int32_t *ids) {
    __shared__ float sh_top[4], sh_sum[4];
    __shared__ int sh_bad;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0) sh_bad = 0;
    for (int j = tid; j < a.k; j += 256) ids[j] = -1;
    __syncthreads();
    float m = -__builtin_inff();
    bool b = false;
    for (int j = tid; j < a.E; j += 256) {
        const float v = load_logit<BF16>(a, t, j);
        row[j] = v;
        b = b || is_bad(v);
        m = fmaxf(m, v);
    }
    m = wave_max_f32(m);
    if (lane == 0) sh_top[wave] = m;
    if (b) sh_bad = 1;
    __syncthreads();
    const float top = fmaxf(fmaxf(sh_top[0], sh_top[1]), fmaxf(sh_top[2], sh_top[3]));
    const bool bad = sh_bad != 0;
    float s = 0.0f;
    if (!bad) {
        for (int j = tid; j < a.E; j += 256) {
            const float v = row[j];
            if (v == -__builtin_inff()) continue;
            int n = 0;
            for (int q = 0; q < a.E; q++) n += (row[q] > v || (row[q] == v && q < j)) ? 1 : 0;
            if (n < a.k) ids[n] = j;
            if (!a.renorm) s += expf(v - top);
        }
    }
    __syncthreads();
    if (a.renorm && !bad && tid < a.k && ids[tid] >= 0) s = expf(row[ids[tid]] - top);
    s = wave_sum_f32(s);
    if (lane == 0) sh_sum[wave] = s;
    __syncthreads();
    const float den = (sh_sum[0] + sh_sum[1]) + (sh_sum[2] + sh_sum[3]);
    if (tid == 0) a.ws_den[t] = bad ? __builtin_nanf("") : den;
    if (tid < a.k) {
        const int e = ids[tid];
        a.ws_ids[t * a.k + tid] = e;
        if (a.ids) a.ids[t * a.k + tid] = e;
        if (a.weights) a.weights[t * a.k + tid] = e >= 0 ? expf(row[e] - top) / den : 0.0f;
    }
}

// One 512-column group of 16 W rows against CT column tiles of 16 activation rows given as bf16 rows
// (arow[c], `planes` planes `plane` elements apart): acc[c] += W . a.  use[c]: whether the lane's row
// takes part (others multiply by zero); any[c]: whether any lane's does (uniform).
template <int CT, int PLANES>
__device__ __forceinline__ void group_product(const MxGroup &w, const __bf16 *const (&arow)[CT], int64_t plane,
                                              const bool (&use)[CT], const bool (&any)[CT], int64_t g, int lg,
                                              int64_t nblk, f32x4 (&acc)[CT]) {
#pragma unroll
    for (int i = 0; i < kGroupChunks; i++) {
        const bool ok = i * 4 + lg < nblk;
        const int64_t blk = g * kGroupBlocks + i * 4 + lg;
        const float s = e8m0_to_f32((w.s[i] >> (8 * lg)) & 255u);
        bf16x8 wf[4];
#pragma unroll
        for (int j = 0; j < 4; j++) wf[j] = fp4_to_bf16x8(w.c[i][j], s);
#pragma unroll
        for (int c = 0; c < CT; c++) {
            if (!any[c]) continue;
#pragma unroll
            for (int p = 0; p < PLANES; p++) {
                u32x4 v[4] = {};
                if (ok && use[c]) {
                    const u32x4 *src = reinterpret_cast<const u32x4 *>(arow[c] + p * plane + blk * kMxBlock);
#pragma unroll
                    for (int j = 0; j < 4; j++) v[j] = src[j];
                }
#pragma unroll
                for (int j = 0; j < 4; j++) acc[c] = mfma_bf16(wf[j], __builtin_bit_cast(bf16x8, v[j]), acc[c]);
            }
        }
    }
}

template <bool LBF16>
__global__ __launch_bounds__(64 * kUpWaves) void k_moe_up(MoeDev a) {
    __shared__ float sh_row[kMaxE];
    __shared__ int32_t sh_ids[kMaxK];
    __shared__ int sh_e, sh_n, sh_rank[kMaxT], sh_tok[kMaxT];
    __shared__ float sh_p[kMaxT];
    __shared__ __align__(16) float red[kUpWaves][2][4][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if ((int)blockIdx.x >= a.slots * a.tiles) {
        route_token<LBF16>(a, blockIdx.x - a.slots * a.tiles, sh_row, sh_ids);
        return;
    }
    const int slot = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
    int e = slot, t0 = 0;
    if (a.pair_slots) {  // the slot's expert: the entry of row t0 with that rank
        t0 = slot / a.k;
        const int want = slot % a.k;
        if (tid == 0) sh_e = -1;
        for (int j = tid; j < a.E; j += 64 * kUpWaves) sh_row[j] = load_logit<LBF16>(a, t0, j);
        __syncthreads();
        for (int j = tid; j < a.E; j += 64 * kUpWaves) {
            const float v = sh_row[j];
            int n = 0;
            for (int q = 0; q < a.E; q++) n += (sh_row[q] > v || (sh_row[q] == v && q < j)) ? 1 : 0;
            if (n == want && v > -__builtin_inff()) sh_e = j;
        }
        __syncthreads();
        e = sh_e;
        if (e < 0) return;
    }
    for (int t = wave; t < a.T; t += kUpWaves) {
        float le, top;
        bool bad;
        const int n = wave_rank<LBF16>(a, t, e, lane, le, top, bad);
        if (lane == 0) {
            sh_rank[t] = (bad || le == -__builtin_inff() || n >= a.k) ? -1 : n;
            sh_p[t] = expf(le - top);
        }
    }
    __syncthreads();
    if (wave == 0) {  // compact the tokens that chose e, in order
        const bool in = lane < a.T && sh_rank[lane] >= 0;
        const uint64_t m = __ballot(in);
        if (in) sh_tok[__popcll(m & ((1ull << lane) - 1))] = lane;
        if (lane == 0) sh_n = __popcll(m);
    }
    __syncthreads();
    const int n = sh_n;
    if (n == 0 || (a.pair_slots && sh_tok[0] != t0)) return;

    const int r = lane & 15, lg = lane >> 4;
    const int64_t kb = a.H / kMxBlock, row = (int64_t)e * 2 * a.I + tile * 16 + r;
    const uint8_t *wc[2], *wsc[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        wc[i] = a.gu_codes + (row + i * a.I) * (a.H / 2);
        wsc[i] = a.gu_scales + (row + i * a.I) * kb;
    }
    const __bf16 *xr[4];
    bool use[4], any[4];
#pragma unroll
    for (int c = 0; c < 4; c++) {
        use[c] = c * 16 + r < n;
        any[c] = c * 16 < n;
        xr[c] = a.x + (int64_t)sh_tok[use[c] ? c * 16 + r : 0] * a.ld_x;
    }
    f32x4 ag[4] = {}, au[4] = {};
    const int64_t ngrp = (a.H + kGroup - 1) / kGroup;
    for (int64_t g = wave; g < ngrp; g += kUpWaves) {
        const int64_t nblk = kb - g * kGroupBlocks;
        const MxGroup wg = load_mx_group(wc[0], wsc[0], g, lg, nblk);
        const MxGroup wu = load_mx_group(wc[1], wsc[1], g, lg, nblk);
        group_product<4, 1>(wg, xr, 0, use, any, g, lg, nblk, ag);
        group_product<4, 1>(wu, xr, 0, use, any, g, lg, nblk, au);
    }
#pragma unroll
    for (int c = 0; c < 4; c++) {
        *reinterpret_cast<f32x4 *>(&red[wave][0][c][lane * 4]) = ag[c];
        *reinterpret_cast<f32x4 *>(&red[wave][1][c][lane * 4]) = au[c];
    }
    __syncthreads();
    for (int o = tid; o < n * 16; o += 64 * kUpWaves) {
        const int il = o % 16, j = o / 16;
        const int at = (j % 16 + 16 * (il / 4)) * 4 + il % 4;
        float gs = 0.0f, us = 0.0f;
#pragma unroll
        for (int w = 0; w < kUpWaves; w++) {
            gs += red[w][0][j / 16][at];
            us += red[w][1][j / 16][at];
        }
        const int t = sh_tok[j];
        const float h = silu(gs) * us * sh_p[t];
        const __bf16 hi = (__bf16)h;
        const int64_t dst = (int64_t)(t * a.k + sh_rank[t]) * a.I + tile * 16 + il;
        a.h_hi[dst] = hi;
        a.h_lo[dst] = (__bf16)(h - (float)hi);
    }
}

template <class OT>
__global__ __launch_bounds__(64 * kDownWaves) void k_moe_down(MoeDev a) {
    __shared__ int sh_ids[kMaxT * kMaxK];
    __shared__ int sh_used[kMaxE], sh_list[kMaxE], sh_nd;
    __shared__ __align__(16) float red[kDownWaves][4][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int pairs = a.T * a.k;
    for (int j = tid; j < a.E; j += 64 * kDownWaves) sh_used[j] = 0;
    __syncthreads();
    for (int j = tid; j < pairs; j += 64 * kDownWaves) {
        const int e = a.ws_ids[j];
        sh_ids[j] = e;
        if (e >= 0) sh_used[e] = 1;
    }
    __syncthreads();
    if (wave == 0) {  // the distinct experts, ascending
        int base = 0;
        for (int j0 = 0; j0 < a.E; j0 += 64) {
            const bool in = j0 + lane < a.E && sh_used[j0 + lane] != 0;
            const uint64_t m = __ballot(in);
            if (in) sh_list[base + __popcll(m & ((1ull << lane) - 1))] = j0 + lane;
            base += __popcll(m);
        }
        if (lane == 0) sh_nd = base;
    }
    __syncthreads();
    const int r = lane & 15, lg = lane >> 4;
    const int64_t kb = a.I / kMxBlock, n0 = (int64_t)blockIdx.x * 16;
    const int64_t ngrp = (a.I + kGroup - 1) / kGroup, items = sh_nd * ngrp;
    const int64_t plane = a.h_lo - a.h_hi;
    f32x4 acc[4] = {};
    for (int64_t it = wave; it < items; it += kDownWaves) {
        const int e = sh_list[it / ngrp];
        const int64_t g = it % ngrp, nblk = kb - g * kGroupBlocks;
        const int64_t row = (int64_t)e * a.H + n0 + r;
        const MxGroup w = load_mx_group(a.dn_codes + row * (a.I / 2), a.dn_scales + row * kb, g, lg, nblk);
        const __bf16 *hr[4];
        bool use[4], any[4];
#pragma unroll
        for (int c = 0; c < 4; c++) {
            const int t = c * 16 + r;
            int at = -1;
            if (t < a.T)
                for (int q = 0; q < a.k; q++)
                    if (sh_ids[t * a.k + q] == e) at = t * a.k + q;
            use[c] = at >= 0;
            any[c] = __any(use[c]);
            hr[c] = a.h_hi + (int64_t)(use[c] ? at : 0) * a.I;
        }
        group_product<4, 2>(w, hr, plane, use, any, g, lg, nblk, acc);
    }
#pragma unroll
    for (int c = 0; c < 4; c++) *reinterpret_cast<f32x4 *>(&red[wave][c][lane * 4]) = acc[c];
    __syncthreads();
    OT *y = reinterpret_cast<OT *>(a.y);
    for (int o = tid; o < a.T * 16; o += 64 * kDownWaves) {
        const int nl = o % 16, t = o / 16;
        const int at = (t % 16 + 16 * (nl / 4)) * 4 + nl % 4;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < kDownWaves; w++) s += red[w][t / 16][at];
        const float den = a.ws_den[t];
        // no expert: 0; a row with NaN or +inf has den = NaN
        const float v = den == 0.0f ? 0.0f : s / den;
        y[(int64_t)t * a.ld_y + n0 + nl] = (OT)v;
    }
}

size_t align256(size_t b) { return (b + 255) / 256 * 256; }

}  // namespace

size_t mx_moe_ws_bytes(int64_t tokens, int64_t top_k, int64_t inter) {
    if (tokens <= 0 || top_k <= 0 || inter < 0) return 0;
    return align256((size_t)tokens * top_k * 4) + align256((size_t)tokens * 4) +
           2 * align256((size_t)tokens * top_k * inter * 2);
}

hipError_t launch_mx_moe(const MoeArgs &p, void *workspace, int num_cus, hipStream_t stream) {
    (void)num_cus;
    MoeDev a{};
    a.x = reinterpret_cast<const __bf16 *>(p.x);
    a.logits = p.logits;
    a.ld_x = p.ld_x;
    a.ld_logits = p.ld_logits;
    a.gu_codes = p.w_gate_up->codes;
    a.gu_scales = p.w_gate_up->scales;
    a.dn_codes = p.w_down->codes;
    a.dn_scales = p.w_down->scales;
    a.H = p.w_gate_up->cols;
    a.I = p.w_down->cols;
    a.y = p.y;
    a.ld_y = p.ld_y;
    a.ids = p.ids;
    a.weights = p.weights;
    a.T = (int)p.tokens;
    a.E = (int)p.experts;
    a.k = p.top_k;
    a.renorm = p.renormalize;
    uint8_t *ws = reinterpret_cast<uint8_t *>(workspace);
    a.ws_ids = reinterpret_cast<int32_t *>(ws);
    ws += align256((size_t)a.T * a.k * 4);
    a.ws_den = reinterpret_cast<float *>(ws);
    ws += align256((size_t)a.T * 4);
    a.h_hi = reinterpret_cast<__bf16 *>(ws);
    a.h_lo = reinterpret_cast<__bf16 *>(ws + align256((size_t)a.T * a.k * a.I * 2));
    a.pair_slots = a.T * a.k < a.E ? 1 : 0;
    a.slots = a.pair_slots ? a.T * a.k : a.E;
    a.tiles = (int)(a.I / 16);
    const dim3 up((unsigned)(a.slots * a.tiles + a.T)), down((unsigned)(a.H / 16));
    if (p.logits_bf16) hipLaunchKernelGGL(k_moe_up<true>, up, dim3(64 * kUpWaves), 0, stream, a);
    else hipLaunchKernelGGL(k_moe_up<false>, up, dim3(64 * kUpWaves), 0, stream, a);
    if (p.y_bf16) hipLaunchKernelGGL(k_moe_down<__bf16>, down, dim3(64 * kDownWaves), 0, stream, a);
    else hipLaunchKernelGGL(k_moe_down<float>, down, dim3(64 * kDownWaves), 0, stream, a);
    return hipGetLastError();
}

}  // namespace nvfp4
