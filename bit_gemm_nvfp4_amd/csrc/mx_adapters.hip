// T = s (A . V^T) of the low-rank adapters of many requests (gfx950): each row of A with the matrix V of its own adapter.
//
// A workgroup takes 16 RM rows of A and 16 RN ranks, and one adapter of those among its rows at a time; the adapters of a
// tile are dealt to blockIdx.z.  Its eight waves split K in chunks of 128 columns and read both operands straight in the
// operand layout of v_mfma_f32_16x16x32_bf16 (a lane's 32 columns of a chunk are contiguous; the order of K is the same on
// both sides), and their sums are joined in LDS in wave order.  V is the first operand, so a lane holds four consecutive
// ranks of one row.  Rows of other adapters are formed too and not stored.
// Few rows: bound by the latency of one pass over V (rank x K x 2 bytes per adapter).  Many: by reading A, and V through L2.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mx_adapters.h"

namespace nvfp4 {

namespace {

constexpr int kDownWaves = 8, kChunk = 128;

struct DownDev {
    const __bf16 *a, *v;
    int64_t lda, M;
    const float *scales;
    const int32_t *index;
    float *t;
    int K, count, rank;
};

// A lane's 32 columns of a chunk, zeros behind the end of the row.
struct Cols {
    u32x4 v[4];
};
__device__ __forceinline__ Cols load_cols(const __bf16 *row, int chunk, int lg, int blocks) {
    Cols c{};
    if (chunk * 4 + lg < blocks) {
        const u32x4 *p = reinterpret_cast<const u32x4 *>(row + chunk * kChunk + lg * kMxBlock);
#pragma unroll
        for (int j = 0; j < 4; j++) c.v[j] = p[j];
    }
    return c;
}

template <int RM, int RN, int AHEAD>
__global__ __launch_bounds__(64 * kDownWaves) void k_adapter_down(DownDev p) {
    __shared__ __align__(16) float red[kDownWaves][RM * RN][256];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, lg = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * RM);
    const int n0 = blockIdx.y * (16 * RN);
    // the adapters of the tile's rows, in the order of their first row; the same in every wave
    const int own = lane < 16 * RM && m0 + lane < p.M ? adapter_of(p.index, p.count, m0 + lane) : -1;
    uint64_t left = __ballot(own >= 0);
    const __bf16 *x[RM];
#pragma unroll
    for (int i = 0; i < RM; i++) x[i] = p.a + min(m0 + 16 * i + r, p.M - 1) * p.lda;
    const int blocks = p.K / kMxBlock, chunks = (p.K + kChunk - 1) / kChunk;
    bool used = false;
    for (int slot = 0; left; slot++) {
        const int a = __builtin_amdgcn_readlane(own, __builtin_ctzll(left));
        const uint64_t rows = __ballot(own == a);
        left &= ~rows;
        if (slot % gridDim.z != blockIdx.z) continue;
        const __bf16 *v[RN];
#pragma unroll
        for (int j = 0; j < RN; j++) v[j] = p.v + ((int64_t)a * p.rank + min(n0 + 16 * j + r, p.rank - 1)) * p.K;
        f32x4 acc[RM][RN] = {};
        for (int c = wave; c < chunks; c += AHEAD * kDownWaves) {
            Cols ca[AHEAD][RM], cv[AHEAD][RN];
#pragma unroll
            for (int q = 0; q < AHEAD; q++) {  // chunks past the last one are zeros
#pragma unroll
                for (int j = 0; j < RN; j++) cv[q][j] = load_cols(v[j], c + q * kDownWaves, lg, blocks);
#pragma unroll
                for (int i = 0; i < RM; i++) ca[q][i] = load_cols(x[i], c + q * kDownWaves, lg, blocks);
            }
#pragma unroll
            for (int q = 0; q < AHEAD; q++)
#pragma unroll
                for (int s = 0; s < 4; s++)
#pragma unroll
                    for (int i = 0; i < RM; i++)
#pragma unroll
                        for (int j = 0; j < RN; j++)
                            acc[i][j] = mfma_bf16(__builtin_bit_cast(bf16x8, cv[q][j].v[s]),
                                                  __builtin_bit_cast(bf16x8, ca[q][i].v[s]), acc[i][j]);
        }
        if (used) __syncthreads();  // the last adapter's sums have been read
        used = true;
#pragma unroll
        for (int i = 0; i < RM; i++)
#pragma unroll
            for (int j = 0; j < RN; j++) *reinterpret_cast<f32x4 *>(&red[wave][i * RN + j][lane * 4]) = acc[i][j];
        __syncthreads();
        const float scale = p.scales ? p.scales[a] : 1.0f;
        // element (rank 4 (l / 16) + q, row l % 16) of a tile sits at 4 l + q; four consecutive ranks per thread
        for (int o = tid; o < RM * RN * 64; o += 64 * kDownWaves) {
            const int tile = o / 64, l = o % 64, row = tile / RN * 16 + l % 16, n = n0 + tile % RN * 16 + l / 16 * 4;
            if (!(rows >> row & 1) || n >= p.rank) continue;  // (rank is a multiple of 8)
            f32x4 s = {};
#pragma unroll
            for (int w = 0; w < kDownWaves; w++) s += *reinterpret_cast<const f32x4 *>(&red[w][tile][l * 4]);
            *reinterpret_cast<f32x4 *>(p.t + (m0 + row) * p.rank + n) = s * scale;
        }
    }
}

template <int RM, int RN, int AHEAD>
void launch_down_t(const DownDev &p, int num_cus, hipStream_t stream) {
    const int64_t tiles = (p.M + 16 * RM - 1) / (16 * RM), cols = (p.rank + 16 * RN - 1) / (16 * RN);
    // as many adapters of a tile side by side as it can have and the device has room for
    const int64_t most = std::min<int64_t>({16 * RM, p.M, p.count}), room = 4 * num_cus / (tiles * cols);
    const dim3 grid((unsigned)tiles, (unsigned)cols, (unsigned)std::max<int64_t>(1, std::min(most, room)));
    hipLaunchKernelGGL((k_adapter_down<RM, RN, AHEAD>), grid, dim3(64 * kDownWaves), 0, stream, p);
}

}  // namespace

hipError_t launch_adapter_down(const AdapterDownArgs &a, int num_cus, hipStream_t stream) {
    const DownDev p{reinterpret_cast<const __bf16 *>(a.a_bf16), reinterpret_cast<const __bf16 *>(a.down), a.lda, a.M, a.scales,
                    a.index, a.t, (int)a.K, a.count, a.rank};
    if (a.M <= 64) launch_down_t<1, 1, 4>(p, num_cus, stream);
    else if (a.rank <= 16) launch_down_t<2, 1, 2>(p, num_cus, stream);
    else if (a.rank <= 32) launch_down_t<2, 2, 1>(p, num_cus, stream);
    else launch_down_t<2, 4, 1>(p, num_cus, stream);
    return hipGetLastError();
}

}  // namespace nvfp4
