// MXFP4 building blocks (E2M1 codes, one E8M0 scale per 32 elements of a row) shared by the mx_*.hip
// kernels, and their host-side launchers.
#pragma once

#include "common.h"
#include "mxfp4.h"

namespace nvfp4 {

constexpr int kMxBlock = 32;

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef u32x4 u32x4_u __attribute__((aligned(1)));  // 16 bytes at any address

// E8M0 byte -> fp32 2^(b - 127): b = 0 is the subnormal 2^-127, b = 255 NaN.
__device__ __forceinline__ float e8m0_to_f32(uint32_t b) {
    const uint32_t u = b == 0 ? 0x00400000u : b << 23;
    return u2f(b == 255 ? 0x7FC00000u : u);
}

// The 32-bit operand of the scaled matrix instructions: four registers of 32 FP4 codes.
__device__ __forceinline__ i32x8 fp4_operand(u32x4 c) {
    return i32x8{(int)c[0], (int)c[1], (int)c[2], (int)c[3], 0, 0, 0, 0};
}

// Rows of 16 (the operand of a 16-row matrix instruction) of an MXFP4 matrix, read straight from
// global memory in groups of kGroup = 512 columns.  Lane l holds row l % 16; in chunk i (128 columns)
// its 16 bytes are block l / 16, which is the operand layout of the 16 x 16 x 128 scaled instruction,
// and a whole row chunk is 64 contiguous bytes.  The 16 scale bytes of a row's group come in one load,
// byte l / 16 of word i being the lane's scale of chunk i.
constexpr int kGroup = 512;
constexpr int kGroupBlocks = kGroup / kMxBlock;
constexpr int kGroupChunks = 4;

struct MxGroup {
    u32x4 c[kGroupChunks];
    u32x4 s;
};

// codes and scales point at the lane's row.
__device__ __forceinline__ MxGroup load_mx_group(const uint8_t *codes, const uint8_t *scales, int grp, int lg) {
    MxGroup r;
    const uint8_t *cp = codes + (int64_t)grp * (kGroup / 2) + lg * 16;
#pragma unroll
    for (int i = 0; i < kGroupChunks; i++) r.c[i] = *reinterpret_cast<const u32x4 *>(cp + i * 64);
    r.s = *reinterpret_cast<const u32x4_u *>(scales + (int64_t)grp * kGroupBlocks);
    return r;
}

// The scale bytes of a partial group (nblk < kGroupBlocks blocks are left); those past the row's end are 0.
__device__ __forceinline__ u32x4 load_mx_tail_scales(const uint8_t *scales, int grp, int nblk) {
    const uint8_t *sp = scales + (int64_t)grp * kGroupBlocks;
    uint32_t s[4] = {0, 0, 0, 0};
    for (int b = 0; b < nblk; b++) {
        const uint32_t v = sp[b];
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (b / 4 == i) s[i] |= v << (8 * (b % 4));
    }
    return u32x4{s[0], s[1], s[2], s[3]};
}

// The last, partial group (nblk < kGroupBlocks blocks are left): blocks past the row's end read as zero
// codes with scale 2^-127.
__device__ __forceinline__ MxGroup load_mx_tail(const uint8_t *codes, const uint8_t *scales, int grp, int lg,
                                                int nblk) {
    MxGroup r;
    const uint8_t *cp = codes + (int64_t)grp * (kGroup / 2) + lg * 16;
#pragma unroll
    for (int i = 0; i < kGroupChunks; i++) {
        r.c[i] = u32x4{0, 0, 0, 0};
        if (i * 4 + lg < nblk) r.c[i] = *reinterpret_cast<const u32x4 *>(cp + i * 64);
    }
    r.s = load_mx_tail_scales(scales, grp, nblk);
    return r;
}

// Eight codes -> eight bf16 values e2m1 x 2^(b - 127), exact.  The scaled conversion reads only the exponent
// field of `scale`, as E8M0: 0 is 2^-127 and 255 NaN; its sign and mantissa do not matter.
__device__ __forceinline__ bf16x8 fp4_to_bf16x8(uint32_t w, float scale) {
    bf16x2 p[4];
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
    return bf16x8{p[0][0], p[0][1], p[1][0], p[1][1], p[2][0], p[2][1], p[3][0], p[3][1]};
}

// Byte `lg` of a word of scale bytes in the exponent field of a conversion scale.
__device__ __forceinline__ float scale_operand(uint32_t word, int lg) {
    return u2f(__builtin_rotateright32(word, 8 * lg + 9));
}

__device__ __forceinline__ f32x4 mfma_bf16(bf16x8 a, bf16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// The bf16 operand of a group: lane l holds block l / 16 of each chunk of row l % 16, 32 values.
struct Bf16Group {
    u32x4 v[kGroupChunks][4];
};

// nblk: blocks of the row from the start of the group on; those past the end read as zero.
template <bool TAIL>
__device__ __forceinline__ Bf16Group load_bf16_group(const __bf16 *row, int grp, int lg, int nblk = kGroupBlocks) {
    Bf16Group r;
    const u32x4 *p = reinterpret_cast<const u32x4 *>(row + (int64_t)grp * kGroup + lg * kMxBlock);
#pragma unroll
    for (int i = 0; i < kGroupChunks; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if constexpr (TAIL) {
                r.v[i][j] = u32x4{0, 0, 0, 0};
                if (i * 4 + lg < nblk) r.v[i][j] = p[i * 16 + j];
            } else {
                r.v[i][j] = p[i * 16 + j];
            }
        }
    return r;
}

// buffer_rsrc with its words forced into scalar registers: a base formed by vector 64-bit arithmetic, though
// the same in every lane, would have each load wrapped in a loop over the lanes' values.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const uint8_t *base, uint32_t bytes) {
    const uint64_t b = reinterpret_cast<uint64_t>(base);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b), hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
    return buffer_rsrc(reinterpret_cast<const uint8_t *>((uint64_t)hi << 32 | lo),
                       (uint32_t)__builtin_amdgcn_readfirstlane(bytes));
}

// acc[t] += W[t] . a over chunk i of a group: the lane's W blocks are expanded exactly to bf16, four instructions
// a tile.  s: the chunk's word of scale bytes of each tile.
template <int RT>
__device__ __forceinline__ void chunk_product(const MxGroup (&w)[RT], const uint32_t (&s)[RT], const Bf16Group &a, int i,
                                              int lg, f32x4 (&acc)[RT]) {
#pragma unroll
    for (int t = 0; t < RT; t++) {
        const float f = scale_operand(s[t], lg);
#pragma unroll
        for (int j = 0; j < 4; j++)
            acc[t] = mfma_bf16(fp4_to_bf16x8(w[t].c[i][j], f), __builtin_bit_cast(bf16x8, a.v[i][j]), acc[t]);
    }
}

template <int RT>
__device__ __forceinline__ void group_product(const MxGroup (&w)[RT], const Bf16Group &a, int lg, f32x4 (&acc)[RT]) {
#pragma unroll
    for (int i = 0; i < kGroupChunks; i++) {
        uint32_t s[RT];
#pragma unroll
        for (int t = 0; t < RT; t++) s[t] = w[t].s[i];
        chunk_product<RT>(w, s, a, i, lg, acc);
    }
}

// Eight fp32 values of a block of 32 that four neighbouring lanes (4 q .. 4 q + 3) hold between them -> the lane's codes
// and the block's scale byte, as mxfp4_quantize makes them.
__device__ __forceinline__ uint32_t mx_encode8(const float (&x)[8], uint32_t &b) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; q++) m = max(m, f2u(x[q]) & 0x7FFFFFFFu);
    m = max(m, dpp_u32<kDppXor1>(m));
    m = max(m, dpp_u32<kDppXor2>(m));
    const uint32_t e = m >> 23;
    b = e == 255 ? 255u : e > 2 ? e - 2 : 0;
    const float inv = u2f((254u - (e > 2 ? e - 2 : 0)) << 23);
    float v[8];
#pragma unroll
    for (int q = 0; q < 8; q++) v[q] = x[q] * inv;
    return e == 255 ? 0u : fp4_pack8(v);
}

// Host side ---------------------------------------------------------------------------------------
hipError_t launch_mx_quantize(const void *x, nvfp4_dtype dt, int64_t ld_x, const float *src_scale,
                              const mxfp4_tensor *out, int32_t *flags, hipStream_t stream);
hipError_t launch_mx_dequantize(const mxfp4_tensor *in, void *out, nvfp4_dtype out_dtype, int64_t ld_out,
                                hipStream_t stream);

// Workspace of mxfp4_gemm: the partial sums of the planned K slices, 0 when unsplit.  first_shape: of the tile shapes.
size_t mx_gemm_ws_bytes(int64_t M, int64_t N, int64_t K, bool a_mx, int num_cus, int first_shape = 0);
hipError_t launch_mx_gemm(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                          void *c, nvfp4_dtype c_dtype, int64_t ldc, void *workspace, size_t workspace_bytes,
                          int num_cus, hipStream_t stream, const struct Adapters *ad = nullptr);

size_t mx_moe_ws_bytes(int64_t pairs, int64_t hidden, int64_t inter);
struct MoeArgs {
    const void *x;
    int64_t tokens, ld_x;
    const void *logits;
    bool logits_bf16;
    int64_t ld_logits, experts;
    int top_k, renormalize;
    const mxfp4_tensor *w_gate_up, *w_down;
    void *y;
    bool y_bf16;
    int64_t ld_y;
    int32_t *ids;
    float *weights;
};
hipError_t launch_mx_moe(const MoeArgs &a, void *workspace, int num_cus, hipStream_t stream);


// Router, sort by group, weighted sum (mx_route.hip).
struct MxRouteArgs {
    const void *logits;
    bool logits_bf16;
    int64_t tokens, ld_logits, experts;
    int top_k, renormalize;
    int32_t *ids;
    float *weights;
    int32_t *offsets, *rows, *places;
};
size_t mx_route_ws_bytes(int64_t tokens, int64_t top_k, int64_t experts);
hipError_t launch_mx_route(const MxRouteArgs &a, void *workspace, hipStream_t stream);
size_t mx_sort_ws_bytes(int64_t pairs, int64_t groups);
// rest: ids outside 0 .. groups - 2 belong to the last group instead of none.
hipError_t launch_mx_sort(const int32_t *ids, int64_t rows, int per_row, int64_t groups, int32_t *offsets, int32_t *out_rows,
                          int32_t *places, bool rest, void *workspace, hipStream_t stream);
hipError_t launch_mx_combine(const void *z, nvfp4_dtype z_dtype, int64_t z_rows, int64_t ld_z, const int32_t *places,
                             const float *weights, int64_t tokens, int top_k, int64_t cols, void *y, nvfp4_dtype y_dtype,
                             int64_t ld_y, hipStream_t stream);

// Products grouped by rows (mx_grouped.hip): C [rows x N] or, with swiglu, [rows x N / 2].
struct MxGroupedArgs {
    const void *a_bf16;         // one of a_bf16 and a_q
    const mxfp4_tensor *a_q;
    int64_t a_rows, lda;
    const int32_t *map;         // row of A of each row of C; null: the same
    const int32_t *offsets;
    int64_t groups, rows;
    const mxfp4_tensor *w;      // [groups * N x K]
    bool swiglu;
    void *c;                    // one of c and c_q (with swiglu)
    nvfp4_dtype c_dtype;
    int64_t ldc;
    const mxfp4_tensor *c_q;
};
hipError_t launch_mx_grouped(const MxGroupedArgs &a, int num_cus, hipStream_t stream);

}  // namespace nvfp4
