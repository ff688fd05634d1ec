// Products with MXFP4 weights whose rows are grouped (gfx950): rows offsets[g] .. offsets[g + 1] - 1 of C are products
// with the weight of group g (an expert), C[i] = A[map[i]] . W[g]^T, with or without silu(gate) * up behind it.
//
// The tiles and their main loop are those of the plain product (mx_tile.h).  A tile never spans two groups, and the
// group sizes are known on the device only, so a launch has as many workgroups as any sizes can need; each finds its
// tile by counting the tiles of the groups before (one wave-wide scan per 64 groups), and those past the last tile end
// at once.  Rows of A are picked by the loads themselves: each lane's offset is its row's.
//
// Gate and up columns: a wave's 64 columns are 32 gate rows of W and the 32 up rows that belong to them, so
// silu(g) * u is formed in the registers of one lane, in fp32, and leaves as fp32, bf16 or MXFP4 (as mxfp4_quantize
// makes it from the fp32 value), without its halves ever being in memory.
//
// What bounds it, kernel times:
//   a few rows per group: streaming the groups' W.  256 rows, 64 groups of which 50 have rows, 4096 x 1536, W4A16 50 us; of W
//     167 MB are needed, 3.3 TB/s, and 176 MB fetched.
//   prompts, W4A16: matrix instructions and the W expansion between them.  4096 rows, 16 groups, gate and up of 4096 x
//     4096 157 us, 0.87 PFLOP/s: about 2.4 rounds of tiles, of which the last is not full, and last tiles of a group that
//     are not.
//   prompts, W4A4: a tile of 256 x 256 takes 3.2 us per 512 columns of K and 8 us for its first loads and its stores.
//     32768 rows, 64 groups, 4096 x 2048 230 to 243 us, 2.3 PFLOP/s.  (A workgroup per CU that works through its tiles
//     and issues the next one's first loads ahead of this one's stores was no faster: all CUs store at a time, 33 MB a
//     round, and the main loop's first wait is for these stores too.)
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mx.h"
#include "mx_tile.h"

namespace nvfp4 {

namespace {

struct GroupedDev {
    const uint8_t *a, *ascales;  // MXFP4 codes and scales, or bf16 rows
    int64_t a_row_bytes, a_row_len;
    int a_rows;
    const int32_t *map, *offsets;
    int groups, rows;
    const uint8_t *wcodes, *wscales;
    int N, K;      // rows and columns of a group's W
    int cols;      // of C: N, or N / 2
    void *c;       // codes for MXFP4
    int64_t ldc;
    uint8_t *cscales;
    int tiles_n, max_tiles_m, vec_c;
    bool stream_w;  // W passes the caches by (MXFP4 A)
};

// Rows lo .. hi - 1 of group g, whatever the offsets hold: within the rows of C.
__device__ __forceinline__ void group_rows(const GroupedDev &p, int g, int &lo, int &hi) {
    lo = max(0, min(p.offsets[g], p.rows));
    hi = max(lo, min(p.offsets[g + 1], p.rows));
}

// The groups' tiles of BM rows, counted 64 groups at a time by each wave.
struct TileScan {
    int lo, hi, upto;  // of the lane's group: its rows, and the tiles up to its end
};

template <int BM>
__device__ __forceinline__ TileScan scan_tiles(const GroupedDev &p, int g0, int before, int lane) {
    TileScan s{0, 0, 0};
    if (g0 + lane < p.groups) group_rows(p, g0 + lane, s.lo, s.hi);
    s.upto = (s.hi - s.lo + BM - 1) / BM;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int v = __shfl_up(s.upto, o);
        if (lane >= o) s.upto += v;
    }
    s.upto += before;
    return s;
}

// A wave's tile of h = silu(g) * u, 32 columns wide, to C [M x cols].
template <class T, class OT>
__device__ __forceinline__ void store_swiglu(uint8_t *lds, const f32x16 (&acc)[T::TM][T::TN], const GroupedDev &p, int64_t row0,
                                             int mw, int M, int nw) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    constexpr int ROW = 40;  // floats between two rows: rows 4 apart start 32 banks apart
    static_assert(T::TN == 2 && ROW <= T::EPI_ROW && (4 * ROW) % 64 == 32, "a gate and an up tile per wave");
    __syncthreads();  // the other waves have read their last operands
    float *buf = reinterpret_cast<float *>(lds + wave * T::EPI_BYTES);
#pragma unroll
    for (int i = 0; i < T::TM; i++) {
#pragma unroll
        for (int e = 0; e < 16; e++) {
            const float g = acc[i][0][e], u = acc[i][1][e];
            buf[(8 * (e / 4) + 4 * h + e % 4) * ROW + (lane & 31)] = g / (1.0f + expf(-g)) * u;
        }
        wave_exchange();
#pragma unroll
        for (int q = 0; q < 2; q++) {  // sixteen rows, eight columns a lane
            const int r = 16 * q + lane / 4, c8 = lane % 4 * 8, m = mw + 32 * i + r, n = nw + c8;
            float v[8];
            *reinterpret_cast<f32x4 *>(v) = *reinterpret_cast<const f32x4 *>(buf + r * ROW + c8);
            *reinterpret_cast<f32x4 *>(v + 4) = *reinterpret_cast<const f32x4 *>(buf + r * ROW + c8 + 4);
            if constexpr (sizeof(OT) == 1) {  // MXFP4: a block is in or out as a whole (cols % 32 == 0)
                uint32_t b;
                const uint32_t w = mx_encode8(v, b);
                if (m < M && nw < p.cols) {
                    *reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(p.c) + (row0 + m) * (p.cols / 2) + n / 2) = w;
                    if (lane % 4 == 0) p.cscales[(row0 + m) * (p.cols / 32) + nw / 32] = (uint8_t)b;
                }
            } else {
                OT *dst = reinterpret_cast<OT *>(p.c) + (row0 + m) * p.ldc + n;
                if (m < M && n + 8 <= p.cols && p.vec_c) {
                    if constexpr (sizeof(OT) == 4) {
                        *reinterpret_cast<f32x4 *>(dst) = f32x4{v[0], v[1], v[2], v[3]};
                        *reinterpret_cast<f32x4 *>(dst + 4) = f32x4{v[4], v[5], v[6], v[7]};
                    } else {
                        *reinterpret_cast<bf16x8 *>(dst) = bf16x8{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3],
                                                                  (__bf16)v[4], (__bf16)v[5], (__bf16)v[6], (__bf16)v[7]};
                    }
                } else if (m < M) {
#pragma unroll
                    for (int j = 0; j < 8; j++)
                        if (n + j < p.cols) store_out(dst + j, v[j]);
                }
            }
        }
        wave_exchange();  // the next rows take their place
    }
}

template <class T, class OT, bool SWIGLU, bool STREAM>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_grouped(GroupedDev p) {
    __shared__ __align__(1024) uint8_t lds[T::LDS_BYTES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // the tile, its group and its rows
    int tiles_m = 0;
    TileScan sc{};
    for (int g0 = 0; g0 < p.groups; g0 += 64) {
        sc = scan_tiles<T::BM>(p, g0, tiles_m, lane);
        tiles_m = __builtin_amdgcn_readlane(sc.upto, 63);
    }
    tiles_m = min(tiles_m, p.max_tiles_m);  // more only if the offsets are not in order
    int tm, tn;
    if (!tile_of(blockIdx.x, tiles_m, p.tiles_n, tm, tn)) return;
    int first = 0, g0 = 0;
    if (p.groups > 64) {
        for (;; g0 += 64) {
            sc = scan_tiles<T::BM>(p, g0, first, lane);
            const int upto = __builtin_amdgcn_readlane(sc.upto, 63);
            if (upto > tm) break;  // there is one: tm < tiles_m
            first = upto;
        }
    }
    const int at = __builtin_ctzll(__ballot(sc.upto > tm));
    const int g = g0 + at, glo = __builtin_amdgcn_readlane(sc.lo, at), ghi = __builtin_amdgcn_readlane(sc.hi, at);
    const int gend = __builtin_amdgcn_readlane(sc.upto, at), gtiles = (ghi - glo + T::BM - 1) / T::BM;
    const int lo = glo + (tm - (gend - gtiles)) * T::BM, mrows = min(T::BM, ghi - lo);

    constexpr int COLS = SWIGLU ? T::BN / 2 : T::BN;  // columns of C
    const int n0 = tn * COLS;
    const int K = p.K;
    // rows of A and W of a tile row, or -1
    auto a_row = [&](int r) -> int {
        if (r >= mrows) return -1;
        if (!p.map) return r;
        const int s = p.map[lo + r];
        return (unsigned)s < (unsigned)p.a_rows ? s : -1;
    };
    auto w_row = [&](int r) -> int {
        if constexpr (SWIGLU) {  // 32 gate rows, then their 32 up rows
            const int col = r / 64 * 32 + r % 32;
            return n0 + col < p.cols ? col + (r & 32 ? p.cols : 0) : -1;
        } else {
            return n0 + r < p.cols ? r : -1;
        }
    };
    const int64_t arow0 = p.map ? 0 : lo, wrow0 = (int64_t)g * p.N + n0;
    const int64_t arows = p.map ? p.a_rows : mrows, wrows = (SWIGLU ? p.cols : 0) + min(COLS, p.cols - n0);
    const MxPicked picked{p.a + arow0 * p.a_row_bytes,
                          p.ascales + arow0 * (K / kMxBlock),
                          arows ? (uint32_t)((arows - 1) * p.a_row_bytes + p.a_row_len) : 0u,
                          (int)p.a_row_bytes,
                          (int)p.a_row_len,
                          p.wcodes + wrow0 * (K / 2),
                          p.wscales + wrow0 * (K / kMxBlock),
                          (uint32_t)(wrows * (K / 2)),
                          K};
    f32x16 acc[T::TM][T::TN] = {};
    mx_picked_product<T, STREAM>(lds, picked, 0, (K + kGroup - 1) / kGroup, a_row, w_row, acc);

    const int mw = wave / T::WN * T::WTM;
    if constexpr (SWIGLU) {
        store_swiglu<T, OT>(lds, acc, p, lo, mw, mrows, n0 + wave % T::WN * 32);
    } else {
        OT *c = reinterpret_cast<OT *>(p.c) + (int64_t)lo * p.ldc;
        mx_store_tile<T>(lds, acc, c, p.ldc, mw, mrows, n0 + wave % T::WN * T::WTN, p.cols, n0 + T::BN <= p.cols && p.vec_c,
                         [](int64_t m, int, int) { return m; });
    }
}

template <class T, class OT, bool SWIGLU>
hipError_t launch_t(GroupedDev p, hipStream_t stream) {
    constexpr int COLS = SWIGLU ? T::BN / 2 : T::BN;
    p.tiles_n = (p.cols + COLS - 1) / COLS;
    p.max_tiles_m = (int)group_tiles(p.rows, p.groups, T::BM);
    const int64_t grid = tile_grid((int64_t)p.max_tiles_m * p.tiles_n);
    if constexpr (T::A_MX && !(T::BM == 128 && T::BN == 128)) {  // (which no streamed product picks)
        if (p.stream_w) {
            hipLaunchKernelGGL((k_mx_grouped<T, OT, SWIGLU, true>), dim3((unsigned)grid), dim3(T::NT), 0, stream, p);
            return hipGetLastError();
        }
    }
    hipLaunchKernelGGL((k_mx_grouped<T, OT, SWIGLU, false>), dim3((unsigned)grid), dim3(T::NT), 0, stream, p);
    return hipGetLastError();
}

template <bool A_MX, class OT, bool SWIGLU>
hipError_t launch_cfg(const GroupedDev &p, int cfg, hipStream_t stream) {
    if constexpr (A_MX) {
        switch (cfg) {
        case 0: return launch_t<MxTile<256, 256, 2, 4, true, 2>, OT, SWIGLU>(p, stream);
        case 1: return launch_t<MxTile<128, 256, 2, 4, true, 3>, OT, SWIGLU>(p, stream);
        case 2: return launch_t<MxTile<128, 128, 4, 2, true, 3>, OT, SWIGLU>(p, stream);
        default: return launch_t<MxTile<64, 128, 2, 2, true, 3>, OT, SWIGLU>(p, stream);
        }
    } else {
        switch (cfg) {
        case 0: return launch_t<MxTile<128, 256, 1, 4, false, 3>, OT, SWIGLU>(p, stream);
        case 1: return launch_t<MxTile<64, 256, 1, 4, false, 3>, OT, SWIGLU>(p, stream);
        case 2: return launch_t<MxTile<32, 256, 1, 4, false, 4>, OT, SWIGLU>(p, stream);
        case 3: return launch_t<MxTile<64, 128, 2, 2, false, 4>, OT, SWIGLU>(p, stream);
        default: return launch_t<MxTile<32, 128, 1, 2, false, 4>, OT, SWIGLU>(p, stream);
        }
    }
}

template <bool A_MX>
hipError_t launch_out(const GroupedDev &p, const MxGroupedArgs &a, int cfg, hipStream_t stream) {
    if (!a.swiglu) {
        if (a.c_dtype == NVFP4_F32) return launch_cfg<A_MX, float, false>(p, cfg, stream);
        return launch_cfg<A_MX, __bf16, false>(p, cfg, stream);
    }
    if (a.c_q) return launch_cfg<A_MX, uint8_t, true>(p, cfg, stream);
    if (a.c_dtype == NVFP4_F32) return launch_cfg<A_MX, float, true>(p, cfg, stream);
    return launch_cfg<A_MX, __bf16, true>(p, cfg, stream);
}

}  // namespace

hipError_t launch_mx_grouped(const MxGroupedArgs &a, int num_cus, hipStream_t stream) {
    GroupedDev p{};
    const bool a_mx = a.a_q != nullptr;
    p.N = (int)(a.w->rows / a.groups);
    p.K = (int)a.w->cols;
    p.a = a_mx ? a.a_q->codes : reinterpret_cast<const uint8_t *>(a.a_bf16);
    p.ascales = a_mx ? a.a_q->scales : nullptr;
    p.a_row_bytes = a_mx ? p.K / 2 : a.lda * 2;
    p.a_row_len = a_mx ? p.K / 2 : p.K * 2;
    p.a_rows = (int)a.a_rows;
    p.map = a.map;
    p.offsets = a.offsets;
    p.groups = (int)a.groups;
    p.rows = (int)a.rows;
    p.wcodes = a.w->codes;
    p.wscales = a.w->scales;
    p.cols = a.swiglu ? p.N / 2 : p.N;
    p.c = a.c_q ? a.c_q->codes : a.c;
    p.cscales = a.c_q ? a.c_q->scales : nullptr;
    p.ldc = a.c_q ? p.cols : a.ldc;
    p.vec_c = reinterpret_cast<uintptr_t>(p.c) % 16 == 0 && p.ldc * (a.c_dtype == NVFP4_F32 ? 4 : 2) % 16 == 0;
    p.stream_w = a_mx && grouped_streams(a.rows, a.groups, p.N, p.K);
    const int cfg = plan_grouped(a.rows, a.groups, p.N, p.K, a_mx, num_cus);
    if (cfg < 0) return hipErrorInvalidConfiguration;
    return a_mx ? launch_out<true>(p, a, cfg, stream) : launch_out<false>(p, a, cfg, stream);
}

}  // namespace nvfp4
