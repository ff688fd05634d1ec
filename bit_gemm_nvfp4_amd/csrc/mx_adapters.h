// The branch of low-rank adapters beside an MXFP4 product (gfx950): row m of C gets s[i] (A[m] . V[i]^T) . U[i]^T of its
// own adapter i = index[m].
//
// T = s (A . V^T) [M x rank] is made first (mx_adapters.hip), as fp32 sums.  The product adds T . U^T to its own sums in
// registers, so C is written once and rounded once:
//   - up to 16 rows: T in fp32, rank multiplications an element;
//   - up to 64, where each row may be a request of its own: the same in a kernel of its own, over all elements side by side,
//     whose fp32 sums the product adds to its own.  (In the product's tiles, one adapter of 32 rows after the other, the
//     branch of 48 x 12288, rank 16, 64 adapters, took 16 us.)
//   - more: T as three bf16 planes that hold the 24 bits of fp32, and matrix instructions.  The product works through the
//     rows in the order of their adapters, so that a tile has few, and takes one of them at a time: U of the tile's columns
//     and T of its rows pass through LDS, 64 ranks at a time.  (Read straight from memory in the operand layout, pieces of
//     16 bytes from 32 rows an instruction, the branch of 4096 x 4096, rank 64, took 20 us.)  T of the
//     others' rows is zero then.  4096 x 4096 x 4096 W4A4, rank 64, 7 requests: 54 us with the product, which takes 38 us alone
//     (44 with rows in another order and no adapter).
//     The order is the sort's, of at most 511 adapters.  With more the rows stay as they come, and a tile of mixed rows has many:
//     the same sizes at random over 511 adapters 343 us, over 512 1524 us; 7 requests of 512 side by side 71 us (80 of 511).
#pragma once

#include "mx_tile.h"

namespace nvfp4 {

constexpr int kAdapterPlanes = 3;
constexpr int64_t kAdapterElementRows = 64;  // T in fp32 up to here; in planes, the rows sorted by adapter, above

struct Adapters {
    const float *t;        // [M x rank], or
    const __bf16 *planes;  // [kAdapterPlanes][M x rank]; rows of no adapter unset
    const float *sums;     // [M x N] the branch, or null; for tiles of up to 64 rows
    const __bf16 *up;      // [count x N x rank]
    const int32_t *index;  // [M]; outside 0 .. count - 1: none
    const int32_t *order;  // [M] the rows in the order of their adapters, and of T's; null: as they are
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

// The adapters of a tile's rows: of the rows 64 i + lane, the same in every wave, and of the rows 32 i + lane % 32 of the
// wave's own; of those also which rows of C they are.  Looked up before the product, whose end does not wait for it then.
template <class T>
struct TileAdapters {
    static constexpr int WORDS = (T::BM + 63) / 64;
    int all[WORDS], mine[T::TM], to[T::TM];
};

template <class T>
__device__ __forceinline__ TileAdapters<T> tile_adapters(const Adapters &ad, int64_t m0, int mrows) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    TileAdapters<T> t;
#pragma unroll
    for (int i = 0; i < TileAdapters<T>::WORDS; i++) {
        const int r = i * 64 + lane;
        t.all[i] = r < mrows ? adapter_of(ad.index, ad.count, ad.order ? ad.order[m0 + r] : m0 + r) : -1;
    }
#pragma unroll
    for (int i = 0; i < T::TM; i++) {
        const int r = wave / T::WN * T::WTM + 32 * i + (lane & 31);
        t.to[i] = r < mrows && ad.order ? ad.order[m0 + r] : r;
        t.mine[i] = r < mrows ? adapter_of(ad.index, ad.count, ad.order ? t.to[i] : m0 + r) : -1;
    }
    return t;
}

// acc += the branch for a tile: rows m0 .. m0 + mrows - 1 of the order, columns n0 .. n0 + nrows - 1.
template <class T>
__device__ __forceinline__ void add_adapters(const Adapters &ad, const TileAdapters<T> &of, uint8_t *lds, f32x16 (&acc)[T::TM][T::TN],
                                             int64_t m0, int mrows, int64_t M, int64_t n0, int nrows, int64_t N) {
    constexpr int T_ROWB = 128, PLANE = T::BM * T_ROWB;  // 64 ranks of a row
    constexpr int U_OFF = kAdapterPlanes * PLANE;
    static_assert(U_OFF + T::BN * T_ROWB <= T::LDS_BYTES, "T and U of a tile");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l32 = lane & 31, h = lane >> 5;
    const int rank = ad.rank, rowb = rank * 2;
    const int mw = wave / T::WN * T::WTM, nw = wave % T::WN * T::WTN;
    if constexpr (T::BM <= kAdapterElementRows) {
        if (ad.sums) {  // the branch's own sums are there
#pragma unroll
            for (int i = 0; i < T::TM; i++)
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const int r = mw + 32 * i + 8 * (e / 4) + 4 * h + e % 4;
                    const float *from = ad.sums + (m0 + min(r, mrows - 1)) * N + n0;  // (rows behind the last are dropped)
#pragma unroll
                    for (int j = 0; j < T::TN; j++) acc[i][j][e] += from[min(nw + 32 * j + l32, nrows - 1)];
                }
            return;
        }
    }
    uint64_t left[TileAdapters<T>::WORDS];
#pragma unroll
    for (int i = 0; i < TileAdapters<T>::WORDS; i++) left[i] = __ballot(of.all[i] >= 0);
    auto next = [&] {  // the adapter of the first row that waits for one, its rows taken out
        int a = -1;
#pragma unroll
        for (int i = 0; i < TileAdapters<T>::WORDS; i++)
            if (a < 0 && left[i]) a = __builtin_amdgcn_readlane(of.all[i], __builtin_ctzll(left[i]));
#pragma unroll
        for (int i = 0; i < TileAdapters<T>::WORDS; i++) left[i] &= ~__ballot(of.all[i] == a);
        return a;
    };
    // A unit of 1 KiB is 8 rows of 128 bytes, swizzled as the product's own.  Rows and ranks that there are not are zeros, and
    // so is T of other adapters' rows.
    // (Whose row it is stands in one word for the rows of a load, and each lane's offsets are those of its first row and whole
    // steps: worked out load by load, a round of one adapter took 8 us, most of it such instructions.)
    constexpr int STEP = T::NW * 8, T_PER = T::BM / STEP, U_PER = T::BN / STEP;  // rows of one load of all waves
    static_assert(T::BM % STEP == 0 && T::BN % STEP == 0 && (STEP == 32 || STEP == 64), "whole loads");
    const uint32_t tbytes = (uint32_t)(mrows * rowb), ubytes = (uint32_t)(nrows * rowb);
    const int ur = wave * 8 + lane / 8, upb = swizzle<8>(ur, lane % 8) * 16;
    __amdgpu_buffer_rsrc_t tr[kAdapterPlanes];
#pragma unroll
    for (int q = 0; q < kAdapterPlanes; q++)
        tr[q] = uniform_rsrc(reinterpret_cast<const uint8_t *>(ad.planes + (q * M + m0) * rank), tbytes);
    auto stage = [&](int a, int k0) {
        const __amdgpu_buffer_rsrc_t u = uniform_rsrc(reinterpret_cast<const uint8_t *>(ad.up + (a * N + n0) * rank), ubytes);
        const uint32_t first = bounds::lane_off((uint32_t)(ur * rowb), k0 * 2, upb, rowb);
        const bool there = first != bounds::kPastRange;
        const uint32_t tsoff = bounds::part_soff(k0 * 2, tbytes), usoff = bounds::part_soff(k0 * 2, ubytes);
#pragma unroll
        for (int i = 0; i < T_PER; i++) {
            const uint64_t own = __ballot(of.all[i * STEP / 64] == a) >> (i * STEP % 64);
            const uint32_t off = there && own >> ur & 1 ? first + (uint32_t)(i * STEP * rowb) : bounds::kPastRange;
#pragma unroll
            for (int q = 0; q < kAdapterPlanes; q++)
                load_to_lds16(tr[q], lds + q * PLANE + (i * T::NW + wave) * 1024, off, tsoff);
        }
#pragma unroll
        for (int i = 0; i < U_PER; i++)
            load_to_lds16(u, lds + U_OFF + (i * T::NW + wave) * 1024, there ? first + (uint32_t)(i * STEP * rowb) : bounds::kPastRange,
                          usoff);
    };
    for (int a; (a = next()) >= 0;) {
        uint64_t bad[T::TN] = {};  // columns (of the lanes) whose U holds an infinity or NaN
        for (int k0 = 0; k0 < rank; k0 += 64) {
            __syncthreads();  // what LDS held has been read
            stage(a, k0);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
            __syncthreads();
            const int slices = min(4, (rank - k0 + 15) / 16);
#pragma unroll 1
            for (int d = 0; d < slices; d++) {
                bf16x8 w[T::TN];
#pragma unroll
                for (int j = 0; j < T::TN; j++) {
                    const int r = nw + 32 * j + l32;
                    u32x4 v = *reinterpret_cast<const u32x4 *>(lds + U_OFF + r * T_ROWB + swizzle<8>(r, 2 * d + h) * 16);
                    bool b = false;
#pragma unroll
                    for (int q = 0; q < 4; q++) b = b || (v[q] & 0x7F80u) == 0x7F80u || (v[q] & 0x7F800000u) == 0x7F800000u;
                    bad[j] |= __ballot(b);
                    w[j] = b ? bf16x8{} : __builtin_bit_cast(bf16x8, v);
                }
#pragma unroll
                for (int i = 0; i < T::TM; i++) {
                    const int r = mw + 32 * i + l32;
                    bf16x8 t[kAdapterPlanes];
#pragma unroll
                    for (int q = 0; q < kAdapterPlanes; q++)
                        t[q] = *reinterpret_cast<const bf16x8 *>(lds + q * PLANE + r * T_ROWB + swizzle<8>(r, 2 * d + h) * 16);
#pragma unroll
                    for (int q = kAdapterPlanes - 1; q >= 0; q--)  // the smallest first
#pragma unroll
                        for (int j = 0; j < T::TN; j++)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(t[q], w[j], acc[i][j], 0, 0, 0);
                }
            }
        }
        // An infinity or NaN in U has been left out, since with T = 0 it would reach other adapters' rows: its column is NaN in
        // the adapter's own.
#pragma unroll
        for (int j = 0; j < T::TN; j++) {
            const uint64_t cols = bad[j] | bad[j] >> 32 | bad[j] << 32;  // (a column's ranks are in two lanes)
            if (cols == 0) continue;
            const bool b = cols >> lane & 1;
#pragma unroll
            for (int i = 0; i < T::TM; i++) {
                const uint32_t rows = (uint32_t)__ballot(of.mine[i] == a);
#pragma unroll
                for (int e = 0; e < 16; e++)
                    acc[i][j][e] = b && rows >> (8 * (e / 4) + 4 * h + e % 4) & 1 ? __builtin_nanf("") : acc[i][j][e];
            }
        }
    }
}

struct MxAdapterTileArgs : MxTileArgs {
    Adapters ad;
};

// The product with the adapters' branch.  Row i of the tiles is row ad.order[i] of A and C where there is an order (rows of
// one adapter side by side), else row i.
template <class T, class OT, bool SPLIT>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_adapter_tile(MxAdapterTileArgs p) {
    __shared__ __align__(1024) uint8_t lds[T::LDS_BYTES];
    int tm, tn;
    if (!tile_of(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn)) return;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m0 = (int64_t)tm * T::BM, n0 = (int64_t)tn * T::BN;
    const int mrows = (int)min((int64_t)T::BM, p.M - m0), nrows = (int)min((int64_t)T::BN, p.N - n0);
    const int K = (int)p.K, wrb = K / 2;
    const int32_t *const order = p.ad.order ? p.ad.order + m0 : nullptr;
    const int64_t base = order ? 0 : m0;  // row of A and C that picked rows count from
    auto a_row = [&](int r) { return r >= mrows ? -1 : order ? order[r] : r; };
    auto w_row = [&](int r) { return r < nrows ? r : -1; };
    const MxPicked picked{p.a + base * p.a_row_bytes,
                          p.ascales + base * (K / kMxBlock),
                          (uint32_t)(((order ? p.M : mrows) - 1) * p.a_row_bytes + p.a_row_len),
                          (int)p.a_row_bytes,
                          (int)p.a_row_len,
                          p.wcodes + n0 * wrb,
                          p.wscales + n0 * (K / kMxBlock),
                          (uint32_t)(nrows * wrb),
                          K};
    const int windows = (K + kGroup - 1) / kGroup;
    const int w0 = (int)blockIdx.y * p.slice_windows, w1 = min(w0 + p.slice_windows, windows);
    const TileAdapters<T> of = tile_adapters<T>(p.ad, m0, mrows);
    f32x16 acc[T::TM][T::TN] = {};
    mx_picked_product<T, false>(lds, picked, w0, w1, a_row, w_row, acc);

    // Of K slices the first has the branch.  (The question stands here without slices too: without it the largest
    // tile's main loop and the branch share a block of code, and registers go to memory.)
    if (blockIdx.y == 0) add_adapters<T>(p.ad, of, lds, acc, m0, mrows, p.M, n0, nrows, p.N);
    OT *c = reinterpret_cast<OT *>(p.c);
    if constexpr (SPLIT) c += (int64_t)blockIdx.y * p.M * p.N;
    const int64_t ldc = SPLIT ? p.N : p.ldc;
    mx_store_tile<T>(lds, acc, c + base * ldc, ldc, wave / T::WN * T::WTM, mrows, n0 + wave % T::WN * T::WTN, p.N,
                     n0 + T::BN <= p.N && p.vec_c, [&](int, int i, int r) -> int64_t { return __shfl(of.to[i], r, 32); });
}

// Host side ---------------------------------------------------------------------------------------
struct AdapterDownArgs {
    const void *a_bf16;
    int64_t M, lda, K;
    const void *down;
    const float *scales;  // may be null
    const int32_t *index, *order;
    int count, rank;
    float *t;        // one of the two forms of T
    __bf16 *planes;
};
hipError_t launch_adapter_down(const AdapterDownArgs &a, int num_cus, hipStream_t stream);
// sums [M x N] = T . U^T
hipError_t launch_adapter_sums(const Adapters &a, int64_t M, int64_t N, float *sums, hipStream_t stream);

}  // namespace nvfp4
