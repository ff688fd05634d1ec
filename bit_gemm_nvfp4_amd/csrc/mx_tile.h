// The tiled MXFP4 product (gfx950): a BM x BN tile of C = A . W^T per workgroup, W MXFP4, A MXFP4 or bf16, with its
// operands passing through LDS.  Shared by the kernels that differ in which rows a tile takes and in what they make of
// the sums.
#pragma once

#include "mx.h"
#include "mx_bounds.h"
#include "mx_plan.h"

namespace nvfp4 {

static_assert(bounds::kPastRange == kOffsetPastRange, "one offset past every range");
static_assert(kPlanWindow == kGroup, "K slices are whole windows of scale bytes");

template <class OT>
__device__ __forceinline__ void store_out(OT *p, float v) {
    *p = (OT)v;
}

// One LDS stage holds BK columns of the tile's rows as they are in memory: 128 bytes of an A row (256 MXFP4
// or 64 bf16 elements) and BK / 2 bytes of a W row, in 16-byte pieces (an MXFP4 block, or 8 bf16 elements).
// Pieces are stored XOR-swizzled by row so that the sixteen consecutive rows of one fragment read spread
// over all banks.
//
// K order: within a step, lanes 0-31 of an operand hold blocks 0 .. KS - 1 and lanes 32-63 blocks KS .. 2 KS - 1,
// KS = BK / 64, so the scale bytes a lane needs for a step are KS consecutive bytes of its row.
//   MXFP4 A: instruction t takes block t of each half, the scale byte picked by its byte select.
//   bf16 A: a lane expands its block of W with the scaled FP4 conversion (exact in bf16, four conversions
//   per eight elements, used by all the wave's A rows) and v_mfma_f32_32x32x16_bf16 q takes elements
//   8 q .. 8 q + 7 of each half's block.  An E4M3 pair per activation would keep W in four bits, but
//   the FP8 matrix instructions align the products of eight elements to 13 bits of the largest, so the
//   sum would lose what the pair carries.
//
// Scale bytes: 16 per row (512 columns, a window) in LDS, two windows; each thread loads its row's next
// window into registers at the start of a window and writes it to LDS at the end.
template <int BM_, int BN_, int WM_, int WN_, bool A_MX_, int NST_>
struct MxTile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr bool A_MX = A_MX_;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int BK = A_MX ? 256 : 64, KS = BK / 64;
    static constexpr int A_ROWB = 128, W_ROWB = BK / 2;
    static constexpr int W_PIECES = W_ROWB / 16;  // 8 or 2
    static constexpr int W_OFF = BM * A_ROWB, STAGE = W_OFF + BN * W_ROWB;
    static constexpr int NST = NST_;
    static constexpr int WINDOW_STEPS = kGroup / BK;
    static constexpr int SA_ROWS = A_MX ? BM : 0, SC_ROWS = SA_ROWS + BN, SC_PER = (SC_ROWS + NT - 1) / NT, SC_OFF = NST * STAGE;
    static constexpr int LDS_BYTES = SC_OFF + 2 * SC_ROWS * 16;
    static constexpr int UNITS = STAGE / 1024, A_UNITS = W_OFF / 1024, UPW = UNITS / NW;
    static constexpr int WTM = BM / WM, WTN = BN / WN, TM = WTM / 32, TN = WTN / 32;
    static constexpr bool WHOLE = TM <= 2;
    static constexpr int READS = TM + (A_MX ? TN : 0);  // LDS reads of a quarter's operands
    // epilogue: 32 rows of a wave's columns; rows 4 apart start 32 banks apart, so that the two halves of a
    // wave write different banks
    static constexpr int EPI_ROW = WTN + 8, EPI_BYTES = 32 * EPI_ROW * 4;
    static_assert((4 * EPI_ROW) % 64 == 32 && NW * EPI_BYTES <= LDS_BYTES, "epilogue rows");
    static_assert(NW % 2 == 0, "the units of a wave share a swizzle");
    static_assert(STAGE % 1024 == 0 && UNITS % NW == 0 && A_UNITS % NW == 0, "tile shape");
    static_assert(LDS_BYTES <= 160 * 1024 && NST >= 2, "LDS stages");
};

// Position of 16-byte piece c of row `row` for rows of `pieces` pieces (8: 128 bytes, 2: 32 bytes): the
// sixteen rows of a fragment read cover the 256 bytes of all banks once.
template <int PIECES>
__device__ __forceinline__ int swizzle(int row, int c) {
    return PIECES == 8 ? c ^ ((row >> 1) & 7) : c ^ ((row >> 3) & 1);
}

// Workgroup id -> tile: ids congruent mod 8 run on one XCD; each XCD gets a contiguous run of tiles in
// bands of kBand tile rows, so that the tiles it works on at a time share A and W rows in its L2.
constexpr int kBand = 4;
__device__ __forceinline__ bool tile_of(int id, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int total = tiles_m * tiles_n, per = (total + 7) / 8;
    const int lin = (id % 8) * per + id / 8;
    if (lin >= total || id / 8 >= per) return false;
    const int band = lin / (kBand * tiles_n), in = lin % (kBand * tiles_n);
    const int h = min(kBand, tiles_m - band * kBand);
    tm = __builtin_amdgcn_readfirstlane(band * kBand + in % h);
    tn = __builtin_amdgcn_readfirstlane(in / h);
    return true;
}

__device__ __forceinline__ u32x4 load_scale_window(const uint8_t *row, int window, int kb) {
    const int nb = kb - window * kGroupBlocks;
    const uint8_t *p = row + window * kGroupBlocks;
    if (nb >= kGroupBlocks) return *reinterpret_cast<const u32x4_u *>(p);
    uint32_t s[4] = {0, 0, 0, 0};
    for (int b = 0; b < nb; b++) {
        const uint32_t v = p[b];
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (b / 4 == i) s[i] |= v << (8 * (b % 4));
    }
    return u32x4{s[0], s[1], s[2], s[3]};
}

// Operands of one quarter of a step, and its matrix instructions.
template <class T>
struct MxFrags {
    u32x4 a[T::TM], w[T::A_MX ? T::TN : 1];
};

// Quarter t: the 64 columns of blocks t and 4 + t (MXFP4 A).
template <class T, int t>
__device__ __forceinline__ void mx_quarter(const MxFrags<T> &f, const int (&sa)[T::TM], const int (&sb)[T::TN],
                                           f32x16 (&acc)[T::TM][T::TN]) {
#pragma unroll
    for (int i = 0; i < T::TM; i++)
#pragma unroll
        for (int j = 0; j < T::TN; j++)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(f.a[i]), fp4_operand(f.w[j]),
                                                                       acc[i][j], 4, 4, t, sa[i], t, sb[j]);
}

// Quarter q: elements 8 q .. 8 q + 7 of the two blocks of a step, W expanded to bf16 (bf16 A).
template <class T>
__device__ __forceinline__ void bf16_quarter(const MxFrags<T> &f, int q, const u32x4 (&w)[T::A_MX ? 1 : T::TN],
                                             const float (&sb)[T::TN], f32x16 (&acc)[T::TM][T::TN]) {
    bf16x8 wf[T::TN];
#pragma unroll
    for (int j = 0; j < T::TN; j++) wf[j] = fp4_to_bf16x8(w[j][q], sb[j]);
#pragma unroll
    for (int i = 0; i < T::TM; i++)
#pragma unroll
        for (int j = 0; j < T::TN; j++)
            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, f.a[i]), wf[j], acc[i][j],
                                                                0, 0, 0);
}

// Keeps the matrix instructions issued so far above this point: the accumulators pass through an empty
// statement.
template <class T>
__device__ __forceinline__ void pin(f32x16 (&acc)[T::TM][T::TN]) {
#pragma unroll
    for (int i = 0; i < T::TM; i++)
#pragma unroll
        for (int j = 0; j < T::TN; j++) asm volatile("" : "+v"(acc[i][j]));
}

// Instruction order of a quarter: two LDS reads behind each of the first matrix instructions, so that the
// next quarter's operands have most of this quarter to arrive in.
template <class T, int READS>
__device__ __forceinline__ void order_quarter() {
#pragma unroll
    for (int r = 0; r < READS / 2; r++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, T::TM * T::TN, 0);
}

// Everything a wave takes from LDS for one step.
template <class T>
struct MxStep {
    MxFrags<T> q[4];
    u32x4 w[T::A_MX ? 1 : T::TN];  // the W blocks (bf16 A)
    int sa[T::TM], sb[T::TN];
};

// Instruction order of a whole step: the LDS reads spread evenly behind its matrix instructions.
template <class T>
__device__ __forceinline__ void order_step() {
    constexpr int M = 4 * T::TM * T::TN;
    constexpr int R = 4 * T::READS + (T::A_MX ? (T::TM + T::TN + 1) / 2 : 2 * T::TN);
    constexpr int PER = (R + M - 1) / M;
#pragma unroll
    for (int i = 0; i < M; i++) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
    }
}

// Main loop, two forms.
// Wave tiles of two 32-row tiles or fewer (T::WHOLE) hold the operands of two whole steps: those of step s + 1
// are read from LDS while the matrix instructions of step s issue, so a read has a whole step to arrive in.
// The step's one barrier stands at its start: stage s + 1 is complete behind it, and stage s, all in
// registers, may be overwritten.
// Taller wave tiles have no registers for that and run in quarters of a step, with the operands of the next
// quarter read while the matrix instructions of this one issue.  The barrier stands before the last quarter,
// whose operands are then in registers: behind it stage s + 1 is complete, so the first operands of step s + 1
// are read under the last quarter's instructions, and stage s may be overwritten.
// W4A16 512 x 4096 x 12288 in quarters: 60.7 us (59.1 in whole steps); W4A4 512 x 12288 x 4096: 25.0 us (23.9).
// What bounds the largest W4A4 tile: a step of 256 columns takes 1.92 us, 1.30 us of them matrix instructions (the
// same loop without anything else) and 1.50 us with the LDS reads; the rest goes to the direct-to-LDS loads, which
// share the LDS with the reads, and the wait at the barrier.
// acc += the product over steps 0 .. nsteps - 1 of a K slice that starts at window w0 of `windows`.  load_stage(s)
// issues the direct-to-LDS loads of step s (T::UPW of them a wave) into stage s % T::NST; srow are the rows of scale
// bytes that the thread serves (null: zeros), kb bytes each.  Returns with no load in flight into LDS; other waves may
// still be reading their last operands.
template <class T, class LoadStage>
__device__ __forceinline__ void mx_tile_product(uint8_t *lds, int kb, int w0, int windows, int nsteps,
                                                const uint8_t *const (&srow)[T::SC_PER], LoadStage load_stage,
                                                f32x16 (&acc)[T::TM][T::TN]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 5;
    u32x4 snext[T::SC_PER];
    auto load_scales = [&](int w) {
#pragma unroll
        for (int i = 0; i < T::SC_PER; i++)
            snext[i] = srow[i] ? load_scale_window(srow[i], w, kb) : u32x4{0, 0, 0, 0};
    };
    auto put_scales = [&](int w) {
#pragma unroll
        for (int i = 0; i < T::SC_PER; i++)
            if (T::SC_ROWS % T::NT == 0 || tid + i * T::NT < T::SC_ROWS)
                *reinterpret_cast<u32x4 *>(lds + T::SC_OFF + (w & 1) * (T::SC_ROWS * 16) + (tid + i * T::NT) * 16) =
                    snext[i];
    };

    const int arow = (wave / T::WN) * T::WTM + (lane & 31), wrow = (wave % T::WN) * T::WTN + (lane & 31);
    // in the order of use: the first matrix instruction takes w[0] and a[0]
    auto read_frags = [&](MxFrags<T> &f, int s, int t) {
        const uint8_t *st = lds + (s % T::NST) * T::STAGE;
        if constexpr (T::A_MX) {  // rows 32 apart have the same swizzle
            const uint8_t *pw = st + T::W_OFF + wrow * T::W_ROWB + swizzle<8>(wrow, 4 * h + t) * 16;
#pragma unroll
            for (int j = 0; j < T::TN; j++) f.w[j] = *reinterpret_cast<const u32x4 *>(pw + j * 32 * T::W_ROWB);
        }
        const uint8_t *pa = st + arow * T::A_ROWB + swizzle<8>(arow, 4 * h + t) * 16;
#pragma unroll
        for (int i = 0; i < T::TM; i++) f.a[i] = *reinterpret_cast<const u32x4 *>(pa + i * 32 * T::A_ROWB);
    };
    // what a whole step needs: scales, and with bf16 A the W blocks
    auto read_step = [&](int s, int (&sa)[T::TM], int (&sb)[T::TN], u32x4 (&wblk)[T::A_MX ? 1 : T::TN]) {
        const uint8_t *sc = lds + T::SC_OFF + ((w0 + s / T::WINDOW_STEPS) & 1) * (T::SC_ROWS * 16);
        const int in = s % T::WINDOW_STEPS;
        if constexpr (T::A_MX) {
#pragma unroll
            for (int i = 0; i < T::TM; i++)
                sa[i] = *reinterpret_cast<const int *>(sc + (arow + 32 * i) * 16 + in * 8 + h * 4);
#pragma unroll
            for (int j = 0; j < T::TN; j++)
                sb[j] = *reinterpret_cast<const int *>(sc + (T::SA_ROWS + wrow + 32 * j) * 16 + in * 8 + h * 4);
        } else {
            const uint8_t *pw = lds + (s % T::NST) * T::STAGE + T::W_OFF + wrow * T::W_ROWB + swizzle<2>(wrow, h) * 16;
#pragma unroll
            for (int j = 0; j < T::TN; j++) {
                sb[j] = sc[(wrow + 32 * j) * 16 + in * 2 + h];
                wblk[j] = *reinterpret_cast<const u32x4 *>(pw + j * 32 * T::W_ROWB);
            }
        }
    };

    load_scales(w0);
    put_scales(w0);
    load_scales(min(w0 + 1, windows - 1));
#pragma unroll
    for (int s = 0; s < T::NST; s++) load_stage(s);
    __builtin_amdgcn_s_waitcnt(waitcnt_imm((T::NST - 1) * T::UPW, 0));
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // The loops' only branches stand before a step's first matrix instruction: with one between them the
    // compiler moves them all behind it, and the operands of the whole step stay live.
    auto next_scales = [&](int s) {
        if (s % T::WINDOW_STEPS == T::WINDOW_STEPS - 1) {
            // the next window's scales, loaded a window ago; their buffer was last read two barriers ago
            const int win = w0 + s / T::WINDOW_STEPS;
            put_scales(win + 1);
            load_scales(min(win + 2, windows - 1));
        }
    };
    auto wait_stage = [&] {
        // the next stage has landed when at most the loads of the NST - 2 later ones are outstanding
        __builtin_amdgcn_s_waitcnt(waitcnt_imm((T::NST - 2) * T::UPW, 0));
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    if constexpr (T::WHOLE) {
        auto read_all = [&](MxStep<T> &f, int s) {
            read_step(s, f.sa, f.sb, f.w);
#pragma unroll
            for (int t = 0; t < 4; t++) read_frags(f.q[t], s, t);
        };
        auto step = [&](int s, const MxStep<T> &cur, MxStep<T> &next) {
            next_scales(s);
            __builtin_amdgcn_sched_barrier(0);
            wait_stage();
            load_stage(s + T::NST);  // past the last step these load zeros or a part that is not read
            read_all(next, s + 1);
            if constexpr (T::A_MX) {
                mx_quarter<T, 0>(cur.q[0], cur.sa, cur.sb, acc);
                mx_quarter<T, 1>(cur.q[1], cur.sa, cur.sb, acc);
                mx_quarter<T, 2>(cur.q[2], cur.sa, cur.sb, acc);
                mx_quarter<T, 3>(cur.q[3], cur.sa, cur.sb, acc);
            } else {
                float sf[T::TN];
#pragma unroll
                for (int j = 0; j < T::TN; j++) sf[j] = scale_operand((uint32_t)cur.sb[j], 0);
#pragma unroll
                for (int t = 0; t < 4; t++) bf16_quarter<T>(cur.q[t], t, cur.w, sf, acc);
            }
            pin<T>(acc);
            order_step<T>();
            __builtin_amdgcn_sched_barrier(0);
        };
        MxStep<T> f0, f1;
        read_all(f0, 0);
        for (int s = 0; s < nsteps; s += 2) {
            step(s, f0, f1);
            if (s + 1 < nsteps) step(s + 1, f1, f0);
        }
    } else {
    int sa[T::TM], sb[T::TN];
    float sf[T::TN];
    u32x4 wblk[T::A_MX ? 1 : T::TN];
    MxFrags<T> f[2];
    read_step(0, sa, sb, wblk);
    read_frags(f[0], 0, 0);
    for (int s = 0; s < nsteps; s++) {
        next_scales(s);
        if constexpr (!T::A_MX) {
#pragma unroll
            for (int j = 0; j < T::TN; j++) sf[j] = scale_operand((uint32_t)sb[j], 0);
        }
        __builtin_amdgcn_sched_barrier(0);
        read_frags(f[1], s, 1);
        if constexpr (T::A_MX) mx_quarter<T, 0>(f[0], sa, sb, acc);
        else bf16_quarter<T>(f[0], 0, wblk, sf, acc);
        pin<T>(acc);
        order_quarter<T, T::READS>();
        __builtin_amdgcn_sched_barrier(0);
        read_frags(f[0], s, 2);
        if constexpr (T::A_MX) mx_quarter<T, 1>(f[1], sa, sb, acc);
        else bf16_quarter<T>(f[1], 1, wblk, sf, acc);
        pin<T>(acc);
        order_quarter<T, T::READS>();
        __builtin_amdgcn_sched_barrier(0);
        read_frags(f[1], s, 3);
        if constexpr (T::A_MX) mx_quarter<T, 2>(f[0], sa, sb, acc);
        else bf16_quarter<T>(f[0], 2, wblk, sf, acc);
        pin<T>(acc);
        order_quarter<T, T::READS>();
        __builtin_amdgcn_sched_barrier(0);
        wait_stage();
        load_stage(s + T::NST);  // past the last step these load zeros or a part that is not read
        int pa[T::TM], pb[T::TN];
        u32x4 pw[T::A_MX ? 1 : T::TN];
#pragma unroll
        for (int i = 0; i < T::TM; i++) pa[i] = sa[i];
#pragma unroll
        for (int j = 0; j < T::TN; j++) pb[j] = sb[j];
#pragma unroll
        for (int j = 0; j < (T::A_MX ? 1 : T::TN); j++) pw[j] = wblk[j];
        read_step(s + 1, sa, sb, wblk);
        read_frags(f[0], s + 1, 0);
        if constexpr (T::A_MX) mx_quarter<T, 3>(f[1], pa, pb, acc);
        else bf16_quarter<T>(f[1], 3, pw, sf, acc);
        pin<T>(acc);
        order_quarter<T, T::READS + (T::A_MX ? (T::TM + T::TN + 1) / 2 : 2 * T::TN)>();
        __builtin_amdgcn_sched_barrier(0);
    }
    }
    // no load may be in flight into the LDS of a workgroup that has ended
    __builtin_amdgcn_s_waitcnt(waitcnt_imm(0, 0));
}

// The wave's sums to C: its corner is (mw, nw) of the M x N matrix c; `wide` where all its columns are there and 16-byte
// stores are aligned.
// row_of(m, i, r): the row of c that row m is, row r of the wave's row tile i; asked by whole waves.
template <class T, class OT, class Row>
__device__ __forceinline__ void mx_store_tile(uint8_t *lds, const f32x16 (&acc)[T::TM][T::TN], OT *c, int64_t ldc, int64_t mw,
                                              int64_t M, int64_t nw, int64_t N, bool wide, Row row_of) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h = lane >> 5;
    constexpr int VEC = 16 / sizeof(OT);
    // Each lane holds single elements of many rows (column l % 32), and a store instruction takes 16
    // cycles whatever its width, so 32 rows at a time pass through LDS (free now, a part per wave) and leave
    // as 16 bytes per lane: a quarter (fp32) or an eighth (bf16) of the stores.  W4A4 4096 x 12288 x 4096 with
    // bf16 C 131 -> 118 us; with fp32 C, which HBM bounds, 133 -> 131 us.
    if (wide) {
        __syncthreads();  // the other waves have read their last operands
        float *buf = reinterpret_cast<float *>(lds + wave * T::EPI_BYTES);
#pragma unroll
        for (int i = 0; i < T::TM; i++) {
#pragma unroll
            for (int e = 0; e < 16; e++)
#pragma unroll
                for (int j = 0; j < T::TN; j++)
                    buf[(8 * (e / 4) + 4 * h + e % 4) * T::EPI_ROW + 32 * j + (lane & 31)] = acc[i][j][e];
            wave_exchange();
            constexpr int LPR = T::WTN / VEC, RPI = 64 / LPR;  // lanes per row, rows per instruction
#pragma unroll
            for (int q = 0; q < 32 / RPI; q++) {
                const int row = q * RPI + lane / LPR, col = lane % LPR * VEC;
                const float *src = buf + row * T::EPI_ROW + col;
                const int64_t m = mw + 32 * i + row, to = row_of(m, i, row);
                if constexpr (VEC == 4) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(src);
                    if (m < M) *reinterpret_cast<f32x4 *>(c + to * ldc + nw + col) = v;
                } else {
                    const f32x4 u = *reinterpret_cast<const f32x4 *>(src), w = *reinterpret_cast<const f32x4 *>(src + 4);
                    const bf16x8 v{(__bf16)u[0], (__bf16)u[1], (__bf16)u[2], (__bf16)u[3],
                                   (__bf16)w[0], (__bf16)w[1], (__bf16)w[2], (__bf16)w[3]};
                    if (m < M) *reinterpret_cast<bf16x8 *>(c + to * ldc + nw + col) = v;
                }
            }
            wave_exchange();  // the next rows take their place
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < T::TM; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) {
            const int row = 8 * (e / 4) + 4 * h + e % 4;
            const int64_t m = mw + 32 * i + row, at = row_of(m, i, row);
            if (m >= M) continue;
            OT *const to = c + at * ldc;
#pragma unroll
            for (int j = 0; j < T::TN; j++) {
                const int64_t n = nw + 32 * j + (lane & 31);
                if (n < N) store_out(to + n, acc[i][j][e]);
            }
        }
}

struct MxTileArgs {
    const uint8_t *a;  // MXFP4 codes or bf16 rows
    const uint8_t *ascales;
    int64_t a_row_bytes, a_row_len;  // distance of two rows of A, and the bytes of a row that are read
    const uint8_t *wcodes, *wscales;
    int64_t M, N, K;
    void *c;
    int64_t ldc;
    int tiles_m, tiles_n;
    int slice_windows;  // windows of 512 columns per K slice (blockIdx.y)
    int vec_c;          // rows of C (of the partial planes) are 16-byte aligned
};

template <class T, class OT, bool SPLIT>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_tile(MxTileArgs p) {
    __shared__ __align__(1024) uint8_t lds[T::LDS_BYTES];
    int tm, tn;
    if (!tile_of(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t m0 = (int64_t)tm * T::BM, n0 = (int64_t)tn * T::BN;
    const int K = (int)p.K, kb = K / kMxBlock;
    const int arb = (int)p.a_row_bytes, wrb = K / 2;  // at most 2^23
    const int alen = (int)p.a_row_len, wlen = wrb;    // bytes of a row
    const int mrows = min(T::BM, (int)p.M - tm * T::BM), nrows = min(T::BN, (int)p.N - tn * T::BN);

    const int windows = (K + kGroup - 1) / kGroup;
    const int w0 = (int)blockIdx.y * p.slice_windows, w1 = min(w0 + p.slice_windows, windows);
    const int step0 = w0 * T::WINDOW_STEPS;
    const int nsteps = min((w1 - w0) * T::WINDOW_STEPS, (K + T::BK - 1) / T::BK - step0);

    // Direct-to-LDS loads: unit u = wave + NW i fills 1 KiB of a stage (8 rows of 128 bytes, or 32 of 32).
    // The units i of all waves have a buffer of their own over the rows that they cover, so the lane
    // part of the offset and the swizzle are the same for all i and the scalar offset is the step's column.  Rows past
    // M or N lie past the buffer's range and load zeros; so do pieces past the end of a row (mx_bounds.h).
    constexpr int A_PER = T::A_UNITS / T::NW, RPU = 64 / T::W_PIECES;
    const int ar = wave * 8 + lane / 8, wr = wave * RPU + lane / T::W_PIECES;
    const int apb = swizzle<8>(ar, lane % 8) * 16, wpb = swizzle<T::W_PIECES>(wr, lane % T::W_PIECES) * 16;
    __amdgpu_buffer_rsrc_t rsrc[T::UPW];
    uint32_t bytes[T::UPW];
#pragma unroll
    for (int i = 0; i < T::UPW; i++) {
        const bool is_a = i < A_PER;
        const bounds::Part part = is_a ? bounds::rows_part(i * (T::NW * 8), T::NW * 8, mrows, arb, alen)
                                       : bounds::rows_part((i - A_PER) * (T::NW * RPU), T::NW * RPU, nrows, wrb, wlen);
        bytes[i] = (uint32_t)__builtin_amdgcn_readfirstlane(part.bytes);
        rsrc[i] = uniform_rsrc((is_a ? p.a + m0 * arb : p.wcodes + n0 * wrb) + part.base, part.bytes);
    }
    auto load_stage = [&](int s) {  // step s of the slice
        uint8_t *dst = lds + (s % T::NST) * T::STAGE + wave * 1024;
        const int ao = (step0 + s) * T::A_ROWB, wo = (step0 + s) * T::W_ROWB;
        const uint32_t av = bounds::lane_off((uint32_t)(ar * arb), ao, apb, alen);
        const uint32_t wv = bounds::lane_off((uint32_t)(wr * wrb), wo, wpb, wlen);
#pragma unroll
        for (int i = 0; i < T::UPW; i++)
            load_to_lds16(rsrc[i], dst + i * (T::NW * 1024), i < A_PER ? av : wv,
                          bounds::part_soff(i < A_PER ? ao : wo, bytes[i]));
    };
    // scale rows [A rows (MXFP4 A), W rows]: thread tid serves rows tid, tid + NT, ...
    const uint8_t *srow[T::SC_PER];
#pragma unroll
    for (int i = 0; i < T::SC_PER; i++) {
        const int r = tid + i * T::NT;
        srow[i] = nullptr;
        if (r < T::SA_ROWS) {
            if (r < mrows) srow[i] = p.ascales + (m0 + r) * (int64_t)kb;
        } else if (r < T::SC_ROWS) {
            if (r - T::SA_ROWS < nrows) srow[i] = p.wscales + (n0 + r - T::SA_ROWS) * (int64_t)kb;
        }
    }
    f32x16 acc[T::TM][T::TN] = {};
    mx_tile_product<T>(lds, kb, w0, windows, nsteps, srow, load_stage, acc);

    OT *c = reinterpret_cast<OT *>(p.c);
    if constexpr (SPLIT) c += (int64_t)blockIdx.y * p.M * p.N;
    const int64_t ldc = SPLIT ? p.N : p.ldc;
    const int64_t mw = m0 + (wave / T::WN) * T::WTM, nw = n0 + (wave % T::WN) * T::WTN;  // the wave's corner
    mx_store_tile<T>(lds, acc, c, ldc, mw, p.M, nw, p.N, n0 + T::BN <= p.N && p.vec_c, [](int64_t m, int, int) { return m; });
}

// The operands of a tile whose rows are picked: a_row(r) and w_row(r) are the rows of tile row r in A and in W, counted from
// a and w, or -1 for none.  Rows lie within a_bytes and w_bytes (below 2^31) of them.
struct MxPicked {
    const uint8_t *a, *ascales;
    uint32_t a_bytes;
    int a_row_bytes, a_row_len;
    const uint8_t *w, *wscales;
    uint32_t w_bytes;
    int K;
};

// load_to_lds16 of lines that the caches let go first.
__device__ __forceinline__ void stream_to_lds16(__amdgpu_buffer_rsrc_t r, void *lds, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)lds, 16, voff, soff, 0, 2);
}

// acc += the product over windows w0 .. w1 - 1 of the tile.  STREAM: W's lines go first where a step takes whole ones (MXFP4 A),
// so that the lines of scale bytes, which eight windows share, stay in L2.
template <class T, bool STREAM, class ARow, class WRow>
__device__ __forceinline__ void mx_picked_product(uint8_t *lds, const MxPicked &p, int w0, int w1, ARow a_row, WRow w_row,
                                                  f32x16 (&acc)[T::TM][T::TN]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int kb = p.K / kMxBlock, wrb = p.K / 2, arb = p.a_row_bytes, alen = p.a_row_len;
    const __amdgpu_buffer_rsrc_t ra = uniform_rsrc(p.a, p.a_bytes), rw = uniform_rsrc(p.w, p.w_bytes);
    const uint32_t abytes = (uint32_t)__builtin_amdgcn_readfirstlane(p.a_bytes),
                   wbytes = (uint32_t)__builtin_amdgcn_readfirstlane(p.w_bytes);
    // Direct-to-LDS loads: unit u = wave + NW i fills 1 KiB of a stage (8 rows of 128 bytes, or 32 of 32).  Every
    // lane's offset is its own row's; those without a row, and pieces past the end of a row, lie past the buffers'
    // ranges and load zeros.
    constexpr int A_PER = T::A_UNITS / T::NW, RPU = 64 / T::W_PIECES;
    const int ar = wave * 8 + lane / 8, wr = wave * RPU + lane / T::W_PIECES;
    const int apb = swizzle<8>(ar, lane % 8) * 16, wpb = swizzle<T::W_PIECES>(wr, lane % T::W_PIECES) * 16;
    uint32_t off[T::UPW];
#pragma unroll
    for (int i = 0; i < T::UPW; i++) {
        const int r = i < A_PER ? a_row(i * (T::NW * 8) + ar) : w_row((i - A_PER) * (T::NW * RPU) + wr);
        off[i] = bounds::row_off(r, i < A_PER ? arb : wrb, i < A_PER ? apb : wpb);
    }
    const int step0 = w0 * T::WINDOW_STEPS;
    auto load_stage = [&](int s) {
        uint8_t *dst = lds + (s % T::NST) * T::STAGE + wave * 1024;
        const int ao = (step0 + s) * T::A_ROWB, wo = (step0 + s) * T::W_ROWB;
        const uint32_t as = bounds::part_soff(ao, abytes), ws = bounds::part_soff(wo, wbytes);
#pragma unroll
        for (int i = 0; i < T::UPW; i++)
            if (i < A_PER)
                load_to_lds16(ra, dst + i * (T::NW * 1024), bounds::step_off(off[i], ao, apb, alen), as);
            else if (STREAM && T::W_ROWB == 128)
                stream_to_lds16(rw, dst + i * (T::NW * 1024), bounds::step_off(off[i], wo, wpb, wrb), ws);
            else
                load_to_lds16(rw, dst + i * (T::NW * 1024), bounds::step_off(off[i], wo, wpb, wrb), ws);
    };
    const uint8_t *srow[T::SC_PER];
#pragma unroll
    for (int i = 0; i < T::SC_PER; i++) {
        const int r = tid + i * T::NT;
        srow[i] = nullptr;
        if (r < T::SA_ROWS) {
            const int s = a_row(r);
            if (s >= 0) srow[i] = p.ascales + (int64_t)s * kb;
        } else if (r < T::SC_ROWS) {
            const int s = w_row(r - T::SA_ROWS);
            if (s >= 0) srow[i] = p.wscales + (int64_t)s * kb;
        }
    }
    const int windows = (p.K + kGroup - 1) / kGroup;
    const int nsteps = min((w1 - w0) * T::WINDOW_STEPS, (p.K + T::BK - 1) / T::BK - step0);
    mx_tile_product<T>(lds, kb, w0, windows, nsteps, srow, load_stage, acc);
}

}  // namespace nvfp4
