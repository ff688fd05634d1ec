// Products with MXFP4 weights for gfx950: C[M x N] = A . W^T, W [N x K] MXFP4, A MXFP4 or bf16.
//
// gfx950's scaled matrix instructions multiply FP4 (or FP8) operands with one E8M0 scale per 32
// elements of K, which is MXFP4 as stored: codes and scale bytes go from memory to the matrix cores
// without any expansion.
//
// k_mx_skinny (M <= 16): bound by streaming W.  A wave reads 16 W rows straight into registers in the
//   operand layout (MxGroup), the waves of a workgroup split K and add their partial tiles in LDS in
//   wave order.  MXFP4 activations take v_mfma_scale_f32_16x16x128; bf16 activations take
//   v_mfma_f32_16x16x32_bf16 on W expanded exactly to bf16 (half an instruction per element), with A staged in
//   LDS.  Calls in a row, W4A16, over weights of 0.8 GB in turn: 1 x 12288 x 4096 7.7 us, 3.5 TB/s of W; 13 x 4096 x
//   12288 12.7 us, where each workgroup's reading of all of A through L2 (320 KB beside 105 KB of W) comes on top of
//   the stream of W.  The same weights again and again, from the Infinity Cache: 6.5 and 10.0 us.  The 16-row bf16 form
//   keeps 45 to 50 scalar values in lanes of vector registers; nothing goes to memory.
// k_mx_tile (M > 16): BM x BN output tile per workgroup, operands through LDS by direct-to-LDS loads,
//   v_mfma_scale_f32_32x32x64 for MXFP4 activations, v_mfma_f32_32x32x16_bf16 for bf16 ones.  4096 x 12288 x
//   4096: W4A4 111 us, 3.7 PFLOP/s; W4A16 321 us, 1.28 PFLOP/s.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include "internal.h"
#include "mx.h"
#include "mx_adapters.h"

namespace nvfp4 {

namespace {

constexpr int kSkinnyMaxM = 16;
static_assert(kTileCost[0][kFirstLowShape].bm <= kAdapterElementRows && kTileCost[1][kFirstLowShape].bm <= kAdapterElementRows &&
                  kTileCost[0][4].bm <= kAdapterElementRows && kTileCost[1][4].bm <= kAdapterElementRows && kTileShapes == 5,
              "tiles that take the branch's sums");
static_assert(kSkinnyMaxM <= kAdapterElementRows, "the form of T that the products of few rows take");
// -------------------------------------------------------------------------------------------------
// M <= 16
// -------------------------------------------------------------------------------------------------
// Bytes between two staged rows of A: sixteen rows start in different banks.
constexpr int kStageRow = kGroup * 2 + 16;

// RT tiles of 16 W rows per wave share its activation operands.  The W groups of a wave are wave, wave +
// waves, ....
//
// MR > 0: bf16 activations, at most MR rows.  A wave stages the rows that a group needs in LDS, a direct-to-LDS load
// of 1 KiB each, one group ahead, with the W groups of the next two in flight.  Read straight in the operand
// layout, each load's 64 lanes would ask for 16-byte pieces of sixteen rows, which the address unit takes piece by
// piece (13 x 4096 x 12288 15.5 -> 11.8 us, 4 rows 10.9 -> 9.0 us).
// MR = 0: MXFP4 activations, a quarter of that, read straight; the next W group's loads are issued before the
// current one's products, into a second set of registers (copied from one set, the copies wait for the loads first: 1 x
// 4096 x 12288 7.5 -> 7.2 us).  The other loop is no faster there (13 x 4096 x 12288 8.9 us, with it 9.8).
// branch(m, n, s): what becomes of the sum s of an element of C before it is rounded.
template <int RT, int MR, class OT, class Branch>
__device__ __forceinline__ void skinny_product(const __bf16 *__restrict__ A, int64_t lda,
                                               const uint8_t *__restrict__ acodes, const uint8_t *__restrict__ ascales,
                                               int M, const uint8_t *__restrict__ wcodes,
                                               const uint8_t *__restrict__ wscales, int64_t N, int K, int stages,
                                               OT *__restrict__ C, int64_t ldc, Branch branch) {
    extern __shared__ __align__(16) float red[];  // [waves][RT][256], then [waves][stages][MR][kStageRow] bytes
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int r = lane & 15, lg = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * (16 * RT);
    const int kb = K / kMxBlock, full = K / kGroup, tail = kb - full * kGroupBlocks;
    // rows past N or M repeat the last one, or are zeros; their results are not stored
    const uint8_t *wc[RT], *ws[RT];
#pragma unroll
    for (int i = 0; i < RT; i++) {
        const int64_t row = min(n0 + 16 * i + r, N - 1);
        wc[i] = wcodes + row * (K / 2);
        ws[i] = wscales + row * kb;
    }
    f32x4 acc[RT] = {};
    if constexpr (MR == 0) {
        const int64_t arow = min(r, M - 1);
        const uint8_t *ac = acodes + arow * (K / 2), *as = ascales + arow * kb;
        auto product = [&](const MxGroup (&w)[RT], const MxGroup &a) {
#pragma unroll
            for (int i = 0; i < kGroupChunks; i++)
#pragma unroll
                for (int t = 0; t < RT; t++)
                    acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        fp4_operand(w[t].c[i]), fp4_operand(a.c[i]), acc[t], 4, 4, 0, (int)(w[t].s[i] >> (8 * lg)), 0,
                        (int)(a.s[i] >> (8 * lg)));
        };
        MxGroup w[2][RT];
        auto load_w = [&](MxGroup (&p)[RT], int g) {
#pragma unroll
            for (int i = 0; i < RT; i++) p[i] = load_mx_group(wc[i], ws[i], g, lg);
        };
        // Group g with the loads of the wave's next one ahead of its products.  Loads return in order: the
        // activations, which come from L2, go ahead of the next W group.
        auto step = [&](const MxGroup (&p)[RT], MxGroup (&next)[RT], int g) {
            const MxGroup a = load_mx_group(ac, as, g, lg);
            __builtin_amdgcn_sched_barrier(0);
            load_w(next, g + waves);
            __builtin_amdgcn_sched_barrier(0);
            product(p, a);
            __builtin_amdgcn_sched_barrier(0);
        };
        if (wave < full) {
            int g = wave;
            load_w(w[0], g);
            for (; g + 2 * waves < full; g += 2 * waves) {
                step(w[0], w[1], g);
                step(w[1], w[0], g + waves);
            }
            if (g + waves < full) {
                step(w[0], w[1], g);
                product(w[1], load_mx_group(ac, as, g + waves, lg));
            } else {
                product(w[0], load_mx_group(ac, as, g, lg));
            }
        }
        if (tail > 0 && full % waves == wave) {
            const MxGroup a = load_mx_tail(ac, as, full, lg, tail);
#pragma unroll
            for (int i = 0; i < RT; i++) w[0][i] = load_mx_tail(wc[i], ws[i], full, lg, tail);
            product(w[0], a);
        }
    } else {
        // Codes of full groups come through a buffer of the workgroup's rows (a row past N repeats the last one);
        // those of groups past the last full one from an empty one.
        const int row_bytes = K / 2, rows = (int)min((int64_t)16 * RT, N - n0);
        uint32_t voff[RT];
#pragma unroll
        for (int t = 0; t < RT; t++) voff[t] = (uint32_t)(min(16 * t + r, rows - 1) * row_bytes + lg * 16);
        auto load_codes = [&](MxGroup (&w)[RT], int g, int i) {
            const uint32_t bytes = g < full ? (uint32_t)(rows * row_bytes) : 0u;
            const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(wcodes + n0 * row_bytes, bytes);
            const uint32_t soff = bounds::part_soff((uint32_t)g * (kGroup / 2), bytes);
#pragma unroll
            for (int t = 0; t < RT; t++)
                w[t].c[i] = __builtin_amdgcn_raw_buffer_load_b128(rw, (int)(voff[t] + i * 64), (int)soff, 0);
        };
        auto load_scales = [&](MxGroup (&w)[RT], int g) {
#pragma unroll
            for (int t = 0; t < RT; t++)
                w[t].s = *reinterpret_cast<const u32x4_u *>(ws[t] + (int64_t)min(g, full - 1) * kGroupBlocks);
        };
        uint8_t *mine = reinterpret_cast<uint8_t *>(red + waves * (RT * 256)) + wave * (stages * MR * kStageRow);
        auto stage = [&](int g, int b) {  // rows past M and columns past K become zeros
            const int bytes = min(kGroup, K - g * kGroup) * 2;
#pragma unroll
            for (int m = 0; m < MR; m++) {
                const __bf16 *row = A + min(m, M - 1) * lda + (int64_t)g * kGroup;
                load_to_lds16(uniform_rsrc(reinterpret_cast<const uint8_t *>(row), m < M && bytes > 0 ? bytes : 0),
                              mine + (b * MR + m) * kStageRow, lane * 16, 0);
            }
            // what arrived() counts as behind these loads stays behind them
            asm volatile("; rows staged" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        // All but the last n loads have arrived, those into LDS among them.  That holds only if the compiled code has
        // n loads between the two marks on every way there; tests/test_mx_waits.py counts them.
        auto arrived = [](auto n) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(waitcnt_imm(n, 15));
            asm volatile("; rows arrived, %0 loads behind" ::"n"(decltype(n)::value) : "memory");
            __builtin_amdgcn_sched_barrier(0);
        };
        auto product = [&](const MxGroup (&w)[RT], int b, int i) {
            const uint8_t *p = mine + (b * MR + r % MR) * kStageRow + lg * 64 + i * 256;
            Bf16Group a;
            uint32_t s[RT];
#pragma unroll
            for (int j = 0; j < 4; j++) a.v[i][j] = *reinterpret_cast<const u32x4 *>(p + j * 16);
#pragma unroll
            for (int t = 0; t < RT; t++) s[t] = w[t].s[i];
            chunk_product<RT>(w, s, a, i, lg, acc);
        };
        // behind the rows of a group come at least the loads of one W group
        constexpr std::integral_constant<int, RT * (kGroupChunks + 1)> behind;
        // One group, with the next one's rows of A behind it, and each chunk's registers taking the chunk of the W
        // group after next as they get free.
        auto step = [&](MxGroup (&p)[RT], int g, int b) {
            arrived(behind);
            stage(min(g + waves, full), b ^ 1);
#pragma unroll
            for (int i = 0; i < kGroupChunks; i++) {
                product(p, b, i);
                __builtin_amdgcn_sched_barrier(0);
                load_codes(p, g + 2 * waves, i);
                __builtin_amdgcn_sched_barrier(0);
            }
            load_scales(p, g + 2 * waves);
            __builtin_amdgcn_sched_barrier(0);
        };
        auto load_w = [&](MxGroup (&p)[RT], int g) {  // in the order of use
            load_scales(p, g);
#pragma unroll
            for (int i = 0; i < kGroupChunks; i++) {
                __builtin_amdgcn_sched_barrier(0);
                load_codes(p, g, i);
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        MxGroup w[2][RT];
        if (wave < full) {
            stage(wave, 0);
            load_w(w[0], wave);
            int g = wave;
            if (g + waves < full) {
                load_w(w[1], g + waves);
                // (two steps in one block: with a way out between them the compiler moves loads of one to the other)
                do {
                    step(w[0], g, 0);
                    step(w[1], g + waves, 1);
                    g += 2 * waves;
                } while (g + waves < full);
            }
            if (g < full) {
                arrived(behind);
#pragma unroll
                for (int i = 0; i < kGroupChunks; i++) product(w[0], 0, i);
            }
        }
        if (tail > 0 && full % waves == wave) {
            __builtin_amdgcn_sched_barrier(0);
            stage(full, 0);
#pragma unroll
            for (int i = 0; i < RT; i++) w[0][i] = load_mx_tail(wc[i], ws[i], full, lg, tail);
            arrived(std::integral_constant<int, 0>());
#pragma unroll
            for (int i = 0; i < kGroupChunks; i++) product(w[0], 0, i);
        }
        // no load may be in flight into the LDS of a workgroup that has ended
        arrived(std::integral_constant<int, 0>());
    }
#pragma unroll
    for (int i = 0; i < RT; i++) *reinterpret_cast<f32x4 *>(&red[(wave * RT + i) * 256 + lane * 4]) = acc[i];
    __syncthreads();
    // element (row nl of the tiles, column m) sits in lane m + 16 (nl % 16 / 4), register nl % 4 of tile nl / 16
    for (int o = threadIdx.x; o < M * 16 * RT; o += blockDim.x) {
        const int nl = o % (16 * RT), m = o / (16 * RT);
        if (n0 + nl >= N) continue;
        const int at = (nl / 16) * 256 + (m + 16 * (nl % 16 / 4)) * 4 + nl % 4;
        float s = 0.0f;
        for (int v = 0; v < waves; v++) s += red[v * (RT * 256) + at];
        store_out(C + (int64_t)m * ldc + n0 + nl, branch(m, n0 + nl, s));
    }
}

template <int RT, int MR, class OT>
__global__ __launch_bounds__(512) void k_mx_skinny(const __bf16 *__restrict__ A, int64_t lda,
                                                   const uint8_t *__restrict__ acodes,
                                                   const uint8_t *__restrict__ ascales, int M,
                                                   const uint8_t *__restrict__ wcodes,
                                                   const uint8_t *__restrict__ wscales, int64_t N, int K, int stages,
                                                   OT *__restrict__ C, int64_t ldc) {
    skinny_product<RT, MR>(A, lda, acodes, ascales, M, wcodes, wscales, N, K, stages, C, ldc,
                           [](int, int64_t, float v) { return v; });
}

// The same with the adapters' branch (mx_adapters.h).
template <int RT, int MR, class OT>
__global__ __launch_bounds__(512) void k_adapter_skinny(const __bf16 *__restrict__ A, int64_t lda,
                                                        const uint8_t *__restrict__ acodes,
                                                        const uint8_t *__restrict__ ascales, int M,
                                                        const uint8_t *__restrict__ wcodes,
                                                        const uint8_t *__restrict__ wscales, int64_t N, int K, int stages,
                                                        OT *__restrict__ C, int64_t ldc, Adapters ad) {
    skinny_product<RT, MR>(A, lda, acodes, ascales, M, wcodes, wscales, N, K, stages, C, ldc,
                           [&](int m, int64_t n, float v) { return v + adapter_value(ad, m, n, N); });
}

// -------------------------------------------------------------------------------------------------
// M > 16
// -------------------------------------------------------------------------------------------------
// The kernels are in mx_tile.h (k_mx_tile) and mx_adapters.h (k_adapter_tile, the product with the adapters' branch).

// C = the sum of the K slices' partial planes, in slice order.  VEC columns per thread (4 where rows of the
// planes and of C allow); the slices' loads are issued together.  Bound by reading the planes.
template <class OT, int VEC>
__global__ __launch_bounds__(256) void k_mx_reduce(const float *__restrict__ P, int splits, int64_t n, uint32_t cols,
                                                   OT *__restrict__ C, int64_t ldc) {
    typedef float vec __attribute__((ext_vector_type(VEC)));
    typedef OT out __attribute__((ext_vector_type(VEC)));
    const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (i >= n) return;
    const float *p = P + i;
    vec s = {};
    for (int k = 0; k < splits; k += 4) {
        vec v[4] = {};
#pragma unroll
        for (int j = 0; j < 4; j++, p += n)
            if (k + j < splits) v[j] = *reinterpret_cast<const vec *>(p);
#pragma unroll
        for (int j = 0; j < 4; j++) s += v[j];
    }
    out o;
#pragma unroll
    for (int q = 0; q < VEC; q++) o[q] = (OT)s[q];
    const int64_t m = n <= 0xFFFFFFFFll ? (uint32_t)i / cols : i / cols;
    *reinterpret_cast<out *>(C + m * ldc + (i - m * cols)) = o;
}

template <class OT>
__global__ __launch_bounds__(256) void k_mx_zero(OT *C, int64_t M, int64_t N, int64_t ldc) {
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * blockDim.x)
        C[(i / N) * ldc + i % N] = (OT)0.0f;
}

// -------------------------------------------------------------------------------------------------
// launches
// -------------------------------------------------------------------------------------------------
template <class T, class OT, bool SPLIT>
void launch_tile_kernel(const MxTileArgs &p, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((k_mx_tile<T, OT, SPLIT>), grid, dim3(T::NT), 0, stream, p);
}
template <class T, class OT, bool SPLIT>
void launch_tile_kernel(const MxAdapterTileArgs &p, dim3 grid, hipStream_t stream) {
    hipLaunchKernelGGL((k_adapter_tile<T, OT, SPLIT>), grid, dim3(T::NT), 0, stream, p);
}

template <class T, class OT, class Args>
void launch_tile_t(Args p, int splits, void *partial, hipStream_t stream) {
    p.tiles_m = (int)((p.M + T::BM - 1) / T::BM);
    p.tiles_n = (int)((p.N + T::BN - 1) / T::BN);
    const dim3 grid((unsigned)tile_grid((int64_t)p.tiles_m * p.tiles_n), splits);
    if (splits == 1) {
        p.vec_c = reinterpret_cast<uintptr_t>(p.c) % 16 == 0 && p.ldc * sizeof(OT) % 16 == 0;
        launch_tile_kernel<T, OT, false>(p, grid, stream);
        return;
    }
    OT *c = reinterpret_cast<OT *>(p.c);
    p.c = partial;
    p.vec_c = p.N % 4 == 0;
    launch_tile_kernel<T, float, true>(p, grid, stream);
    const int64_t n = p.M * p.N;
    const float *planes = reinterpret_cast<const float *>(partial);
    if (p.vec_c && reinterpret_cast<uintptr_t>(c) % (4 * sizeof(OT)) == 0 && p.ldc % 4 == 0)
        hipLaunchKernelGGL((k_mx_reduce<OT, 4>), dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, planes,
                           splits, n, (uint32_t)p.N, c, p.ldc);
    else
        hipLaunchKernelGGL((k_mx_reduce<OT, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, planes, splits,
                           n, (uint32_t)p.N, c, p.ldc);
}

template <class OT, class Args>
hipError_t launch_tiled(Args p, int first_shape, const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                        OT *c, int64_t ldc, void *workspace, size_t workspace_bytes, int num_cus, hipStream_t stream) {
    p.M = M;
    p.N = w->rows;
    p.K = w->cols;
    p.wcodes = w->codes;
    p.wscales = w->scales;
    p.c = c;
    p.ldc = ldc;
    const bool a_mx = a_q != nullptr;
    p.a = a_mx ? a_q->codes : reinterpret_cast<const uint8_t *>(a_bf16);
    p.ascales = a_mx ? a_q->scales : nullptr;
    p.a_row_bytes = a_mx ? p.K / 2 : lda * 2;
    p.a_row_len = a_mx ? p.K / 2 : p.K * 2;
    const MxPlan plan = plan_mx_within(M, p.N, p.K, a_mx, num_cus, workspace ? workspace_bytes : 0, first_shape);
    if (plan.cfg < 0) return hipErrorInvalidConfiguration;
    p.slice_windows = plan.slice_windows;
    if (a_mx) {
        switch (plan.cfg) {
        case 0: launch_tile_t<MxTile<256, 256, 2, 4, true, 2>, OT>(p, plan.splits, workspace, stream); break;
        case 1: launch_tile_t<MxTile<128, 256, 2, 4, true, 3>, OT>(p, plan.splits, workspace, stream); break;
        case 2: launch_tile_t<MxTile<128, 128, 4, 2, true, 3>, OT>(p, plan.splits, workspace, stream); break;
        case 3: launch_tile_t<MxTile<64, 64, 2, 2, true, 3>, OT>(p, plan.splits, workspace, stream); break;
        default: launch_tile_t<MxTile<64, 128, 2, 2, true, 3>, OT>(p, plan.splits, workspace, stream); break;
        }
    } else {
        switch (plan.cfg) {
        case 0: launch_tile_t<MxTile<256, 256, 2, 4, false, 3>, OT>(p, plan.splits, workspace, stream); break;
        case 1: launch_tile_t<MxTile<128, 256, 2, 4, false, 3>, OT>(p, plan.splits, workspace, stream); break;
        case 2: launch_tile_t<MxTile<128, 128, 2, 2, false, 3>, OT>(p, plan.splits, workspace, stream); break;
        case 3: launch_tile_t<MxTile<64, 128, 1, 4, false, 4>, OT>(p, plan.splits, workspace, stream); break;
        default: launch_tile_t<MxTile<32, 128, 1, 4, false, 4>, OT>(p, plan.splits, workspace, stream); break;
        }
    }
    return hipGetLastError();
}

// ad: null for the product without adapters.
template <int RT, int MR, class OT>
void launch_skinny_t(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w, OT *c,
                     int64_t ldc, int waves, int stages, const Adapters *ad, hipStream_t stream) {
    const unsigned wgs = (unsigned)((w->rows + 16 * RT - 1) / (16 * RT));
    const size_t lds = (size_t)waves * (RT * 1024 + stages * MR * kStageRow);
    const __bf16 *a = reinterpret_cast<const __bf16 *>(a_bf16);
    const uint8_t *ac = a_q ? a_q->codes : nullptr, *as = a_q ? a_q->scales : nullptr;
    if (ad)
        hipLaunchKernelGGL((k_adapter_skinny<RT, MR, OT>), dim3(wgs), dim3(64 * waves), lds, stream, a, lda, ac, as, (int)M,
                           w->codes, w->scales, w->rows, (int)w->cols, stages, c, ldc, *ad);
    else
        hipLaunchKernelGGL((k_mx_skinny<RT, MR, OT>), dim3(wgs), dim3(64 * waves), lds, stream, a, lda, ac, as, (int)M,
                           w->codes, w->scales, w->rows, (int)w->cols, stages, c, ldc);
}

// W row tiles per workgroup and its waves.  Every workgroup reads all of A through L2 (16 rows of bf16 are 3.8
// times a tile of W), so tiles share it, as many as spread over the CUs in one round, up to three (four
// spill).  Measured, us (K = 4096 unless said, weights of up to 0.6 GB in turn), with 1, 2 and 3 tiles, the pick marked:
//   bf16  1 x 12288: 9.0, 10.0, 7.5 *;  16 x 12288: 13.9, 12.9, 9.6 *;  16 x 12288, K = 12288: 35.8, 32.9, 24.5 *
//   bf16  16 x 6000: 8.9, 6.9 *, 8.2;  8 x 8192: 7.9, 6.9 *, 7.3
//   bf16  16 x 4096: 5.4 *, 6.6, 8.0;  13 x 4096, K = 12288: 11.8 *, 15.9, 20.7
//   MXFP4 1 x 12288: 7.4, 8.0, 7.0 *;  16 x 12288: 9.6, 10.0, 8.2 *;  16 x 6000: 7.0, 6.2 *, 7.3
//   MXFP4 16 x 4096: 4.8 *, 6.0, 7.2;  13 x 4096, K = 12288: 8.9 *, 12.3, 15.6
// Waves split K.  MXFP4: 8 with three tiles (2 and 4 waves 11.3, 11.4 against 11.1), else 4 (8 x 8192: 2, 4, 8 waves
// 7.3, 7.4, 7.6).  bf16, up to 8 rows: 8 where three tiles make one round (1 x 12288 8.3, with 4 8.8), else 4 (1 x
// 50000 29.5, with 8 34.8).  bf16, 16 rows: 8 where one stage of A per wave is enough (16 x 4096 5.8, with 4 6.3);
// two fit in LDS only four times.
template <int MR, class OT>
void launch_skinny(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w, OT *c,
                   int64_t ldc, int num_cus, const Adapters *ad, hipStream_t stream) {
    const int64_t tiles = (w->rows + 15) / 16, groups = (w->cols + kGroup - 1) / kGroup;
    const int64_t share = (tiles + num_cus - 1) / num_cus;
    int waves = (MR == 0 ? share >= 3 : MR == 16 ? groups <= 8 : share == 3) ? 8 : 4;
    while (waves > 1 && waves / 2 >= groups) waves /= 2;  // no more waves than groups to share out
    const int stages = groups > waves ? 2 : 1;
    if (share >= 3) launch_skinny_t<3, MR, OT>(a_bf16, a_q, M, lda, w, c, ldc, waves, stages, ad, stream);
    else if (share == 2) launch_skinny_t<2, MR, OT>(a_bf16, a_q, M, lda, w, c, ldc, waves, stages, ad, stream);
    else launch_skinny_t<1, MR, OT>(a_bf16, a_q, M, lda, w, c, ldc, waves, stages, ad, stream);
}

template <class OT>
hipError_t launch_mx_gemm_t(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                            OT *c, int64_t ldc, void *workspace, size_t workspace_bytes, int num_cus, const Adapters *ad,
                            hipStream_t stream) {
    if (w->cols == 0) {
        const int64_t blocks = std::min<int64_t>((M * w->rows + 255) / 256, 4096);
        hipLaunchKernelGGL(k_mx_zero<OT>, dim3((unsigned)blocks), dim3(256), 0, stream, c, M, w->rows, ldc);
    } else if (M <= kSkinnyMaxM) {
        if (a_q) launch_skinny<0>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, ad, stream);
        else if (M <= 4) launch_skinny<4>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, ad, stream);
        else if (M <= 8) launch_skinny<8>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, ad, stream);
        else launch_skinny<16>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, ad, stream);
    } else if (ad) {
        return launch_tiled(MxAdapterTileArgs{{}, *ad}, ad->sums ? kFirstLowShape : 0, a_bf16, a_q, M, lda, w, c, ldc, workspace, workspace_bytes, num_cus, stream);
    } else {
        return launch_tiled(MxTileArgs{}, 0, a_bf16, a_q, M, lda, w, c, ldc, workspace, workspace_bytes, num_cus, stream);
    }
    return hipGetLastError();
}

}  // namespace

size_t mx_gemm_ws_bytes(int64_t M, int64_t N, int64_t K, bool a_mx, int num_cus, int first_shape) {
    if (M <= kSkinnyMaxM || N <= 0 || K <= 0) return 0;
    return plan_ws_bytes(plan_mx(M, N, K, a_mx, num_cus, kMaxSplits, first_shape), M, N);
}

hipError_t launch_mx_gemm(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                          void *c, nvfp4_dtype c_dtype, int64_t ldc, void *workspace, size_t workspace_bytes,
                          int num_cus, hipStream_t stream, const Adapters *ad) {
    if (c_dtype == NVFP4_F32)
        return launch_mx_gemm_t(a_bf16, a_q, M, lda, w, reinterpret_cast<float *>(c), ldc, workspace, workspace_bytes,
                                num_cus, ad, stream);
    return launch_mx_gemm_t(a_bf16, a_q, M, lda, w, reinterpret_cast<__bf16 *>(c), ldc, workspace, workspace_bytes,
                            num_cus, ad, stream);
}

}  // namespace nvfp4
