// T = s (A . V^T) of the low-rank adapters of many requests (gfx950): each row of A with the matrix V of its own adapter.
//
// A workgroup takes 16 RM rows of A and 16 RN ranks, and one adapter of those among its rows at a time; the adapters of a
// tile are dealt to blockIdx.z.  Both operands pass through LDS by direct-to-LDS loads, NW 32 columns at a time, whole
// pieces of rows per load; wave w multiplies its 32 columns of each chunk (v_mfma_f32_16x16x32_bf16), and the waves' sums are
// joined in LDS in wave order.  V is the first operand, so a lane holds four consecutive ranks of one row.  Rows of other
// adapters are formed too and not stored.
// (Read straight in the operand layout, 16-byte pieces of sixteen rows, a load of 1 KiB took about 70 cycles of the address
// unit: 4096 x 4096, rank 64, 25 us; 1 x 4096, rank 16, 6.3 us.)
// Few rows: bound by the latency of one pass over V (rank x K x 2 bytes per adapter): 1 x 4096, rank 16 4.5 us, 48 rows of 64
// adapters 6.8 us.  Many: by A and V coming through L2: 4096 x 4096, rank 64 16 us.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "internal.h"
#include "mx_adapters.h"

namespace nvfp4 {

namespace {

struct DownDev {
    const __bf16 *a, *v;
    int64_t lda, M;
    const float *scales;
    const int32_t *index, *order;
    float *t;
    __bf16 *planes;
    int K, count, rank;
};

template <int RM, int RN, int NW, int NST>
__global__ __launch_bounds__(64 * NW) void k_adapter_down(DownDev p) {
    constexpr int ROWB = NW * 64, RPU = 16 / NW, LPR = 4 * NW;  // bytes of a row's chunk; rows of 1 KiB; lanes of a row
    constexpr int LOADS = RM + RN, STAGE = LOADS * NW * 1024;   // a wave's loads per chunk: its part of each 16 rows
    __shared__ __align__(1024) uint8_t lds[NST * STAGE];
    static_assert(NW * RM * RN * 1024 <= NST * STAGE && NST >= 3, "the waves' sums; stages");
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, lg = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * (16 * RM);
    const int n0 = blockIdx.y * (16 * RN), rowlen = p.K * 2;
    auto row_of = [&](int64_t m) -> int64_t { return p.order ? p.order[m] : m; };
    // the adapters of the tile's rows, in the order of their first row; the same in every wave
    const int own = lane < 16 * RM && m0 + lane < p.M ? adapter_of(p.index, p.count, row_of(m0 + lane)) : -1;
    uint64_t left = __ballot(own >= 0);
    // rows of A in another order are picked from all of it (below 2^31 bytes), else from the tile's own
    const int64_t base = p.order ? 0 : m0, have = p.order ? p.M : min((int64_t)16 * RM, p.M - m0);
    const int vrows = min(16 * RN, p.rank - n0);
    const uint32_t xbytes = (uint32_t)((have - 1) * p.lda * 2 + rowlen), vbytes = (uint32_t)(vrows * rowlen);
    const __amdgpu_buffer_rsrc_t xr = uniform_rsrc(reinterpret_cast<const uint8_t *>(p.a + base * p.lda), xbytes);
    // the wave's rows, and its 16-byte piece of them: XOR-swizzled so that sixteen rows of one piece lie in different banks
    const int wr = wave * RPU + lane / LPR, at = ((lane % LPR) ^ (wr & 15)) * 16;
    uint32_t off[LOADS];
#pragma unroll
    for (int i = 0; i < LOADS; i++) {
        if (i < RM) {
            const int64_t m = m0 + 16 * i + wr;
            off[i] = m < p.M ? (uint32_t)((row_of(m) - base) * p.lda * 2 + at) : bounds::kPastRange;
        } else {
            off[i] = bounds::row_off(16 * (i - RM) + wr < vrows ? 16 * (i - RM) + wr : -1, rowlen, at);
        }
    }
    const int chunks = (rowlen + ROWB - 1) / ROWB;
    bool used = false;
    for (int slot = 0; left; slot++) {
        const int a = __builtin_amdgcn_readlane(own, __builtin_ctzll(left));
        const uint64_t rows = __ballot(own == a);
        left &= ~rows;
        if (slot % gridDim.z != blockIdx.z) continue;
        const __amdgpu_buffer_rsrc_t vr =
            uniform_rsrc(reinterpret_cast<const uint8_t *>(p.v + ((int64_t)a * p.rank + n0) * p.K), vbytes);
        auto load = [&](int c) {  // chunks past the last one, and pieces past the end of a row, are zeros
            uint8_t *dst = lds + (c % NST) * STAGE + wave * 1024;
#pragma unroll
            for (int i = 0; i < LOADS; i++)
                load_to_lds16(i < RM ? xr : vr, dst + i * (NW * 1024), bounds::step_off(off[i], c * ROWB, at, rowlen),
                              bounds::part_soff((uint32_t)(c * ROWB), i < RM ? xbytes : vbytes));
        };
        if (used) __syncthreads();  // the last adapter's sums have been read
        used = true;
        f32x4 acc[RM][RN] = {};
#pragma unroll
        for (int c = 0; c < NST - 1; c++) load(c);
        for (int c = 0; c < chunks; c++) {
            // chunk c has landed when at most the loads of the NST - 2 later ones are outstanding; the one before it has been
            // read by all waves behind the barrier
            __builtin_amdgcn_s_waitcnt(waitcnt_imm((NST - 2) * LOADS, 0));
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            load(c + NST - 1);
            const uint8_t *st = lds + (c % NST) * STAGE + r * ROWB + ((wave * 4 + lg) ^ r) * 16;
            bf16x8 x[RM], v[RN];
#pragma unroll
            for (int i = 0; i < RM; i++) x[i] = *reinterpret_cast<const bf16x8 *>(st + i * (16 * ROWB));
#pragma unroll
            for (int j = 0; j < RN; j++) v[j] = *reinterpret_cast<const bf16x8 *>(st + (RM + j) * (16 * ROWB));
#pragma unroll
            for (int i = 0; i < RM; i++)
#pragma unroll
                for (int j = 0; j < RN; j++) acc[i][j] = mfma_bf16(v[j], x[i], acc[i][j]);
            __builtin_amdgcn_sched_barrier(0);
        }
        __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));  // nothing is in flight into the sums' place
        __syncthreads();
        float *red = reinterpret_cast<float *>(lds);  // [wave][tile][256]
#pragma unroll
        for (int i = 0; i < RM; i++)
#pragma unroll
            for (int j = 0; j < RN; j++)
                *reinterpret_cast<f32x4 *>(red + (wave * (RM * RN) + i * RN + j) * 256 + lane * 4) = acc[i][j];
        __syncthreads();
        const float scale = p.scales ? p.scales[a] : 1.0f;
        // element (rank 4 (l / 16) + q, row l % 16) of a tile sits at 4 l + q; four consecutive ranks per thread
        for (int o = tid; o < RM * RN * 64; o += 64 * NW) {
            const int tile = o / 64, l = o % 64, row = tile / RN * 16 + l % 16, n = n0 + tile % RN * 16 + l / 16 * 4;
            if (!(rows >> row & 1) || n >= p.rank) continue;  // (rank is a multiple of 8)
            f32x4 s = {};
#pragma unroll
            for (int w = 0; w < NW; w++) s += *reinterpret_cast<const f32x4 *>(red + (w * (RM * RN) + tile) * 256 + l * 4);
            s *= scale;
            const int64_t to = (m0 + row) * p.rank + n;
            if (p.t) {
                *reinterpret_cast<f32x4 *>(p.t + to) = s;
            } else {
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                bf16x4 part[kAdapterPlanes];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    __bf16 hi, mid, lo;
                    three_planes(s[i], hi, mid, lo);
                    part[0][i] = hi;
                    part[1][i] = mid;
                    part[2][i] = lo;
                }
#pragma unroll
                for (int q = 0; q < kAdapterPlanes; q++) *reinterpret_cast<bf16x4 *>(p.planes + q * p.M * p.rank + to) = part[q];
            }
        }
    }
}

// The branch's sums, a column of C per thread and a row per blockIdx.y.
__global__ __launch_bounds__(256) void k_adapter_sums(Adapters ad, int64_t N, float *__restrict__ sums) {
    const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, m = blockIdx.y;
    if (n < N) sums[m * N + n] = adapter_value(ad, m, n, N);
}

template <int RM, int RN, int NW, int NST>
void launch_down_t(const DownDev &p, int num_cus, hipStream_t stream) {
    const int64_t tiles = (p.M + 16 * RM - 1) / (16 * RM), cols = (p.rank + 16 * RN - 1) / (16 * RN);
    // as many adapters of a tile side by side as it can have and the device has room for
    const int64_t most = std::min<int64_t>({16 * RM, p.M, p.count}), room = 4 * num_cus / (tiles * cols);
    const dim3 grid((unsigned)tiles, (unsigned)cols, (unsigned)std::max<int64_t>(1, std::min(most, room)));
    hipLaunchKernelGGL((k_adapter_down<RM, RN, NW, NST>), grid, dim3(64 * NW), 0, stream, p);
}

}  // namespace

hipError_t launch_adapter_down(const AdapterDownArgs &a, int num_cus, hipStream_t stream) {
    const DownDev p{reinterpret_cast<const __bf16 *>(a.a_bf16), reinterpret_cast<const __bf16 *>(a.down), a.lda, a.M, a.scales,
                    a.index, a.order, a.t, a.planes, (int)a.K, a.count, a.rank};
    // Few tiles: small ones, with more of K side by side.  The operator in microseconds, 16 x 16 in 256 columns and the other form
    // (K = 4096, C 32 wide): 48 rows, rank 16 16.3 and 18.7; 512 rows, rank 64 24.8 and 34.4; 4096 rows, rank 16 38.9 and 37.9,
    // rank 32 44.8 and 41.2, rank 64 54.6 and 45.7, rank 128 75.7 and 55.7.
    if (a.M <= 1024) launch_down_t<1, 1, 8, 4>(p, num_cus, stream);
    else if (a.rank <= 16) launch_down_t<2, 1, 4, 4>(p, num_cus, stream);
    else if (a.rank <= 32) launch_down_t<2, 2, 4, 4>(p, num_cus, stream);
    else launch_down_t<2, 4, 4, 3>(p, num_cus, stream);
    return hipGetLastError();
}

hipError_t launch_adapter_sums(const Adapters &a, int64_t M, int64_t N, float *sums, hipStream_t stream) {
    hipLaunchKernelGGL(k_adapter_sums, dim3((unsigned)((N + 255) / 256), (unsigned)M), dim3(256), 0, stream, a, N, sums);
    return hipGetLastError();
}

}  // namespace nvfp4
