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
#include "mx_bounds.h"
#include "mx_plan.h"

namespace nvfp4 {

namespace {

constexpr int kSkinnyMaxM = 16;
static_assert(bounds::kPastRange == kOffsetPastRange, "one offset past every range");
static_assert(kPlanWindow == kGroup, "K slices are whole windows of scale bytes");

template <class OT>
__device__ __forceinline__ void store_out(OT *p, float v) {
    *p = (OT)v;
}

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
template <int RT, int MR, class OT>
__global__ __launch_bounds__(512) void k_mx_skinny(const __bf16 *__restrict__ A, int64_t lda,
                                                   const uint8_t *__restrict__ acodes,
                                                   const uint8_t *__restrict__ ascales, int M,
                                                   const uint8_t *__restrict__ wcodes,
                                                   const uint8_t *__restrict__ wscales, int64_t N, int K, int stages,
                                                   OT *__restrict__ C, int64_t ldc) {
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
        store_out(C + (int64_t)m * ldc + n0 + nl, s);
    }
}

// -------------------------------------------------------------------------------------------------
// M > 16
// -------------------------------------------------------------------------------------------------
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
template <class T, class OT, bool SPLIT>
__global__ __launch_bounds__(T::NT) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_mx_tile(MxTileArgs p) {
    __shared__ __align__(1024) uint8_t lds[T::LDS_BYTES];
    int tm, tn;
    if (!tile_of(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn)) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = lane >> 5;
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

    f32x16 acc[T::TM][T::TN] = {};
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

    OT *c = reinterpret_cast<OT *>(p.c);
    if constexpr (SPLIT) c += (int64_t)blockIdx.y * p.M * p.N;
    const int64_t ldc = SPLIT ? p.N : p.ldc;
    const int64_t mw = m0 + (wave / T::WN) * T::WTM, nw = n0 + (wave % T::WN) * T::WTN;  // the wave's corner
    constexpr int VEC = 16 / sizeof(OT);
    // Each lane holds single elements of many rows (column l % 32), and a store instruction takes 16
    // cycles whatever its width, so 32 rows at a time pass through LDS (free now, a part per wave) and leave
    // as 16 bytes per lane: a quarter (fp32) or an eighth (bf16) of the stores.  W4A4 4096 x 12288 x 4096 with
    // bf16 C 131 -> 118 us; with fp32 C, which HBM bounds, 133 -> 131 us.
    if (n0 + T::BN <= p.N && p.vec_c) {
        __syncthreads();  // the other waves have read their last operands
        float *buf = reinterpret_cast<float *>(lds + wave * T::EPI_BYTES);
#pragma unroll
        for (int i = 0; i < T::TM; i++) {
#pragma unroll
            for (int e = 0; e < 16; e++)
#pragma unroll
                for (int j = 0; j < T::TN; j++)
                    buf[(8 * (e / 4) + 4 * h + e % 4) * T::EPI_ROW + 32 * j + (lane & 31)] = acc[i][j][e];
            constexpr int LPR = T::WTN / VEC, RPI = 64 / LPR;  // lanes per row, rows per instruction
#pragma unroll
            for (int q = 0; q < 32 / RPI; q++) {
                const int row = q * RPI + lane / LPR, col = lane % LPR * VEC;
                const float *src = buf + row * T::EPI_ROW + col;
                const int64_t m = mw + 32 * i + row;
                if constexpr (VEC == 4) {
                    const f32x4 v = *reinterpret_cast<const f32x4 *>(src);
                    if (m < p.M) *reinterpret_cast<f32x4 *>(c + m * ldc + nw + col) = v;
                } else {
                    const f32x4 u = *reinterpret_cast<const f32x4 *>(src), w = *reinterpret_cast<const f32x4 *>(src + 4);
                    const bf16x8 v{(__bf16)u[0], (__bf16)u[1], (__bf16)u[2], (__bf16)u[3],
                                   (__bf16)w[0], (__bf16)w[1], (__bf16)w[2], (__bf16)w[3]};
                    if (m < p.M) *reinterpret_cast<bf16x8 *>(c + m * ldc + nw + col) = v;
                }
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < T::TM; i++)
#pragma unroll
        for (int e = 0; e < 16; e++) {
            const int64_t m = mw + 32 * i + 8 * (e / 4) + 4 * h + e % 4;
            if (m >= p.M) continue;
#pragma unroll
            for (int j = 0; j < T::TN; j++) {
                const int64_t n = nw + 32 * j + (lane & 31);
                if (n < p.N) store_out(c + m * ldc + n, acc[i][j][e]);
            }
        }
}

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
template <class T, class OT>
void launch_tile_t(MxTileArgs p, int splits, void *partial, hipStream_t stream) {
    p.tiles_m = (int)((p.M + T::BM - 1) / T::BM);
    p.tiles_n = (int)((p.N + T::BN - 1) / T::BN);
    const dim3 grid((unsigned)tile_grid((int64_t)p.tiles_m * p.tiles_n), splits);
    if (splits == 1) {
        p.vec_c = reinterpret_cast<uintptr_t>(p.c) % 16 == 0 && p.ldc * sizeof(OT) % 16 == 0;
        hipLaunchKernelGGL((k_mx_tile<T, OT, false>), grid, dim3(T::NT), 0, stream, p);
        return;
    }
    OT *c = reinterpret_cast<OT *>(p.c);
    p.c = partial;
    p.vec_c = p.N % 4 == 0;
    hipLaunchKernelGGL((k_mx_tile<T, float, true>), grid, dim3(T::NT), 0, stream, p);
    const int64_t n = p.M * p.N;
    const float *planes = reinterpret_cast<const float *>(partial);
    if (p.vec_c && reinterpret_cast<uintptr_t>(c) % (4 * sizeof(OT)) == 0 && p.ldc % 4 == 0)
        hipLaunchKernelGGL((k_mx_reduce<OT, 4>), dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, stream, planes,
                           splits, n, (uint32_t)p.N, c, p.ldc);
    else
        hipLaunchKernelGGL((k_mx_reduce<OT, 1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, planes, splits,
                           n, (uint32_t)p.N, c, p.ldc);
}

template <class OT>
hipError_t launch_tiled(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w, OT *c,
                        int64_t ldc, void *workspace, size_t workspace_bytes, int num_cus, hipStream_t stream) {
    MxTileArgs p{};
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
    const MxPlan plan = plan_mx_within(M, p.N, p.K, a_mx, num_cus, workspace ? workspace_bytes : 0);
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

template <int RT, int MR, class OT>
void launch_skinny_t(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w, OT *c,
                     int64_t ldc, int waves, int stages, hipStream_t stream) {
    const unsigned wgs = (unsigned)((w->rows + 16 * RT - 1) / (16 * RT));
    const size_t lds = (size_t)waves * (RT * 1024 + stages * MR * kStageRow);
    hipLaunchKernelGGL((k_mx_skinny<RT, MR, OT>), dim3(wgs), dim3(64 * waves), lds, stream,
                       reinterpret_cast<const __bf16 *>(a_bf16), lda, a_q ? a_q->codes : nullptr,
                       a_q ? a_q->scales : nullptr, (int)M, w->codes, w->scales, w->rows, (int)w->cols, stages, c, ldc);
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
                   int64_t ldc, int num_cus, hipStream_t stream) {
    const int64_t tiles = (w->rows + 15) / 16, groups = (w->cols + kGroup - 1) / kGroup;
    const int64_t share = (tiles + num_cus - 1) / num_cus;
    int waves = (MR == 0 ? share >= 3 : MR == 16 ? groups <= 8 : share == 3) ? 8 : 4;
    while (waves > 1 && waves / 2 >= groups) waves /= 2;  // no more waves than groups to share out
    const int stages = groups > waves ? 2 : 1;
    if (share >= 3) launch_skinny_t<3, MR, OT>(a_bf16, a_q, M, lda, w, c, ldc, waves, stages, stream);
    else if (share == 2) launch_skinny_t<2, MR, OT>(a_bf16, a_q, M, lda, w, c, ldc, waves, stages, stream);
    else launch_skinny_t<1, MR, OT>(a_bf16, a_q, M, lda, w, c, ldc, waves, stages, stream);
}

template <class OT>
hipError_t launch_mx_gemm_t(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                            OT *c, int64_t ldc, void *workspace, size_t workspace_bytes, int num_cus,
                            hipStream_t stream) {
    if (w->cols == 0) {
        const int64_t blocks = std::min<int64_t>((M * w->rows + 255) / 256, 4096);
        hipLaunchKernelGGL(k_mx_zero<OT>, dim3((unsigned)blocks), dim3(256), 0, stream, c, M, w->rows, ldc);
    } else if (M <= kSkinnyMaxM) {
        if (a_q) launch_skinny<0>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, stream);
        else if (M <= 4) launch_skinny<4>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, stream);
        else if (M <= 8) launch_skinny<8>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, stream);
        else launch_skinny<16>(a_bf16, a_q, M, lda, w, c, ldc, num_cus, stream);
    } else {
        return launch_tiled(a_bf16, a_q, M, lda, w, c, ldc, workspace, workspace_bytes, num_cus, stream);
    }
    return hipGetLastError();
}

}  // namespace

size_t mx_gemm_ws_bytes(int64_t M, int64_t N, int64_t K, bool a_mx, int num_cus) {
    if (M <= kSkinnyMaxM || N <= 0 || K <= 0) return 0;
    return plan_ws_bytes(plan_mx(M, N, K, a_mx, num_cus), M, N);
}

hipError_t launch_mx_gemm(const void *a_bf16, const mxfp4_tensor *a_q, int64_t M, int64_t lda, const mxfp4_tensor *w,
                          void *c, nvfp4_dtype c_dtype, int64_t ldc, void *workspace, size_t workspace_bytes,
                          int num_cus, hipStream_t stream) {
    if (c_dtype == NVFP4_F32)
        return launch_mx_gemm_t(a_bf16, a_q, M, lda, w, reinterpret_cast<float *>(c), ldc, workspace, workspace_bytes,
                                num_cus, stream);
    return launch_mx_gemm_t(a_bf16, a_q, M, lda, w, reinterpret_cast<__bf16 *>(c), ldc, workspace, workspace_bytes,
                            num_cus, stream);
}

}  // namespace nvfp4
