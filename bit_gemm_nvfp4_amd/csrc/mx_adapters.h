// The branch of low-rank adapters beside an MXFP4 product (gfx950): row m of C gets s[i] (A[m] . V[i]^T) . U[i]^T of its
// own adapter i = index[m].
//
// T = s (A . V^T) [M x rank] is made first (mx_adapters.hip), in fp32.  The product adds T . U^T to its sums in registers,
// so C is written once and rounded once:
//   - up to 16 rows: fp32 sums, rank multiplications an element;
//   - more rows: matrix instructions.  T goes in as three bf16 planes that hold the 24 bits of fp32, and the rows of a tile
//     are taken one adapter at a time: the sums of all its rows are formed, and those of the adapter's own are added.
//     (Zeros in place of the others' T would do as well, but for an adapter that holds an infinity or NaN, which then
//     would reach rows of others.)
#pragma once

#include "mx.h"

namespace nvfp4 {

struct Adapters {
    const float *t;        // [M x rank], rows of no adapter unset
    const __bf16 *up;      // [count x N x rank]
    const int32_t *index;  // [M]; outside 0 .. count - 1: none
    int count, rank;
};

__device__ __forceinline__ int adapter_of(const int32_t *index, int count, int64_t m) {
    const int a = index[m];
    return (unsigned)a < (unsigned)count ? a : -1;
}

// T[m] . U[n] of m's adapter.
__device__ __forceinline__ float adapter_value(const Adapters &ad, int64_t m, int64_t n, int64_t N) {
    const int a = adapter_of(ad.index, ad.count, m);
    float s = 0.0f;
    if (a < 0) return s;
    const u32x4 *u = reinterpret_cast<const u32x4 *>(ad.up + (a * N + n) * ad.rank);
    const f32x4 *t = reinterpret_cast<const f32x4 *>(ad.t + m * ad.rank);
    for (int k = 0; k < ad.rank / 8; k++) {
        const u32x4 w = u[k];
        const f32x4 t0 = t[2 * k], t1 = t[2 * k + 1];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t v = w[i];
            s += (i < 2 ? t0[2 * i] : t1[2 * i - 4]) * u2f(v << 16);
            s += (i < 2 ? t0[2 * i + 1] : t1[2 * i - 3]) * u2f(v & 0xFFFF0000u);
        }
    }
    return s;
}

// fp32 as three bf16 planes, cut off, so that none rounds beyond bf16's range; an infinity or NaN has no rest.
__device__ __forceinline__ void three_planes(float v, __bf16 &hi, __bf16 &mid, __bf16 &lo) {
    const bool finite = (f2u(v) & 0x7F800000u) != 0x7F800000u;
    const float h = u2f(f2u(v) & 0xFFFF0000u), rest = finite ? v - h : 0.0f, m = u2f(f2u(rest) & 0xFFFF0000u);
    hi = (__bf16)(finite ? h : v);
    mid = (__bf16)m;
    lo = (__bf16)(rest - m);
}

// acc += the branch for a wave's sums, whose corner is (mw, nw) of C [M x N].
template <int TM, int TN>
__device__ __forceinline__ void add_adapters(const Adapters &ad, f32x16 (&acc)[TM][TN], int64_t mw, int64_t M, int64_t nw,
                                             int64_t N) {
    const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5, rank = ad.rank;
    int own[TM];
    uint32_t left[TM];  // rows that still wait for their adapter
#pragma unroll
    for (int i = 0; i < TM; i++) {
        const int64_t m = mw + 32 * i + l32;
        own[i] = m < M ? adapter_of(ad.index, ad.count, m) : -1;
        left[i] = (uint32_t)__ballot(own[i] >= 0);
    }
    for (;;) {
        int a = -1;
#pragma unroll
        for (int i = 0; i < TM; i++)
            if (a < 0 && left[i]) a = __builtin_amdgcn_readlane(own[i], __builtin_ctz(left[i]));
        if (a < 0) break;
        const __bf16 *u[TN];
#pragma unroll
        for (int j = 0; j < TN; j++) u[j] = ad.up + (a * N + min(nw + 32 * j + l32, N - 1)) * rank + 8 * h;
#pragma unroll
        for (int i = 0; i < TM; i++) {
            const uint32_t rows = (uint32_t)__ballot(own[i] == a);
            if (rows == 0) continue;
            left[i] &= ~rows;
            const float *t = ad.t + min(mw + 32 * i + l32, M - 1) * rank + 8 * h;
            f32x16 sum[TN] = {};
            for (int k = 0; k < rank; k += 16) {
                bf16x8 p[3] = {}, w[TN] = {};
                if (k + 8 * h < rank) {
                    const f32x4 t0 = *reinterpret_cast<const f32x4 *>(t + k), t1 = *reinterpret_cast<const f32x4 *>(t + k + 4);
#pragma unroll
                    for (int q = 0; q < 8; q++) {
                        __bf16 x0, x1, x2;
                        three_planes(q < 4 ? t0[q] : t1[q - 4], x0, x1, x2);
                        p[0][q] = x0;
                        p[1][q] = x1;
                        p[2][q] = x2;
                    }
#pragma unroll
                    for (int j = 0; j < TN; j++) w[j] = *reinterpret_cast<const bf16x8 *>(u[j] + k);
                }
#pragma unroll
                for (int j = 0; j < TN; j++)
#pragma unroll
                    for (int q = 2; q >= 0; q--)  // the smallest first
                        sum[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(p[q], w[j], sum[j], 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 16; e++) {
                const bool mine = rows >> (8 * (e / 4) + 4 * h + e % 4) & 1;
#pragma unroll
                for (int j = 0; j < TN; j++) acc[i][j][e] += mine ? sum[j][e] : 0.0f;
            }
            // one tile of rows after the other: side by side they need more registers than there are
#pragma unroll
            for (int j = 0; j < TN; j++) asm volatile("" : "+v"(acc[i][j]));
            __builtin_amdgcn_sched_barrier(0);
        }
    }
}

// Host side ---------------------------------------------------------------------------------------
struct AdapterDownArgs {
    const void *a_bf16;
    int64_t M, lda, K;
    const void *down;
    const float *scales;  // may be null
    const int32_t *index;
    int count, rank;
    float *t;
};
hipError_t launch_adapter_down(const AdapterDownArgs &a, int num_cus, hipStream_t stream);

}  // namespace nvfp4
