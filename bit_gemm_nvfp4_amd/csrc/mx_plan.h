// Tile shape and K slices of an MXFP4 product of more than 16 rows, by a measured cost.  Free of HIP types, so that
// host code can ask for the plan of any size.
#pragma once

#include <stdint.h>

namespace nvfp4 {

constexpr int kMaxSplits = 8;     // K slices of a tiled product
constexpr int kPlanWindow = 512;  // columns that a slice is a multiple of

struct MxPlan {
    int cfg;            // index into the tile shapes, -1 when the tiles of none fit one launch
    int splits;         // K slices
    int slice_windows;  // windows of 512 columns per slice
};

// Tile shapes and what they cost: microseconds per tile (start, first loads, stores) and per window of 512
// columns, with one workgroup per CU and with `per_cu` of them.  Fitted to timings of every shape with 1, 2
// and 4 K slices on an MI355X; of those, in microseconds (tile: time; the shape picked is marked):
//   W4A4   512 x 12288 x 4096   256x256: 33.1   128x256: 23.9 *  128x128: 30.3   64x128: 29.8   64x64: 36.6
//   W4A4   512 x 4096 x 12288   128x256: 53.4   128x128: 34.7 (two slices: 31.4)   64x128: 27.7 *  64x64: 32.4
//   W4A4   4096 x 4096 x 4096   256x256: 40.1 * 128x256: 45.2    128x128: 54.1
//   W4A4   1024 x 4096 x 4096   128x256: 20.2   128x128: 15.6 *  64x128: 18.6   64x64: 22.9
//   W4A4   256 x 4096 x 4096    128x256: 18.7   128x128: 12.8    64x128: 10.0   64x64: 8.7 *
//   W4A16  512 x 12288 x 4096   256x256: 81.4   128x256: 50.1 *  128x128: 55.5   64x128: 60.3
//   W4A16  512 x 4096 x 12288   128x256: 128.4, in four slices 59.1 *  128x128 in two: 64.2
//   W4A16  128 x 4096 x 4096    128x128: 35.6   64x128: 24.6, in four slices 16.9 *  32x128 in two: 17.3
//   W4A16  17 x 12288 x 4096    64x128: 24.7, in four slices 16.6   32x128: 21.0, in four slices 14.8 *
//   W4A16  4096 x 12288 x 4096  256x256: 313 *  128x256: 359     128x128: 361
struct TileCost {
    int bm, bn, waves, per_cu;
    double start, window, window_full;
};
constexpr int kTileShapes = 5;
constexpr TileCost kTileCost[2][kTileShapes] = {
    {{256, 256, 8, 1, 3.0, 12.6, 12.6},
     {128, 256, 8, 1, 5.0, 6.4, 6.4},
     {128, 128, 4, 2, 4.0, 4.0, 7.0},
     {64, 128, 4, 2, 3.0, 2.8, 4.5},
     {32, 128, 4, 2, 3.0, 2.1, 3.0}},
    {{256, 256, 8, 1, 7.8, 3.84, 3.84},
     {128, 256, 8, 1, 5.0, 2.4, 2.4},
     {128, 128, 8, 1, 2.5, 1.5, 1.5},
     {64, 64, 4, 2, 2.4, 0.82, 1.2},
     {64, 128, 4, 2, 2.5, 1.05, 1.8}},
};
constexpr uint64_t kMaxGridThreads = 0xFFFFFFFFull;  // of one launch, in x
constexpr double kReduceStart = 4.0, kReduceBytesPerUs = 3.0e6;  // the pass that adds the slices

// Workgroups of a product's tiles: whole rounds over the eight XCDs.
inline int64_t tile_grid(int64_t tiles) { return (tiles + 7) / 8 * 8; }

constexpr int kFirstLowShape = 3;  // the shapes from here on are at most 64 rows high

// The cheapest of the shapes from `first` on and of up to `max_splits` K slices.
inline MxPlan plan_mx(int64_t M, int64_t N, int64_t K, bool a_mx, int num_cus, int max_splits = kMaxSplits, int first = 0) {
    const int64_t windows = (K + kPlanWindow - 1) / kPlanWindow;
    MxPlan best{-1, 1, (int)windows};
    double cost = 1e30;
    for (int cfg = first; cfg < kTileShapes; cfg++) {
        const TileCost &t = kTileCost[a_mx ? 1 : 0][cfg];
        const int64_t tiles = ((M + t.bm - 1) / t.bm) * ((N + t.bn - 1) / t.bn);
        if ((uint64_t)tile_grid(tiles) * 64 * t.waves > kMaxGridThreads) continue;
        for (int64_t s = 1; s <= max_splits && s <= windows; s++) {
            const int64_t per = (windows + s - 1) / s;
            if ((windows + per - 1) / per != s) continue;  // a slice would be empty
            const int64_t all = tiles * s, slots = (int64_t)num_cus * t.per_cu;
            double us = all <= num_cus ? t.start + per * t.window
                                       : (double)((all + slots - 1) / slots) * (t.start + per * t.window_full);
            if (s > 1) us += kReduceStart + (double)M * N * 4 * (s + 1) / kReduceBytesPerUs;
            if (us < cost) {
                cost = us;
                best = MxPlan{cfg, (int)s, (int)per};
            }
        }
    }
    return best;
}

inline uint64_t plan_ws_bytes(const MxPlan &p, int64_t M, int64_t N) {
    return p.splits > 1 ? (uint64_t)p.splits * (uint64_t)M * (uint64_t)N * 4 : 0;
}

// The plan that runs with a workspace of `have` bytes: the cheapest, or the cheapest without K slices where that one's
// partial sums do not fit (W4A16 512 x 4096 x 12288 without a workspace: 128x256, the shape of the four slices, 128 us;
// 64x128 72.5 us).
inline MxPlan plan_mx_within(int64_t M, int64_t N, int64_t K, bool a_mx, int num_cus, uint64_t have, int first = 0) {
    const MxPlan p = plan_mx(M, N, K, a_mx, num_cus, kMaxSplits, first);
    return plan_ws_bytes(p, M, N) <= have ? p : plan_mx(M, N, K, a_mx, num_cus, 1, first);
}

// Products grouped by rows: tile shapes of 64 columns a wave (a gate and an up tile of 32), and their costs as above,
// fitted to timings of every shape at 64 sizes (8 to 32768 rows, 1 to 128 groups of uneven sizes) on an MI355X, where the
// shape picked is within 1.3 % of the fastest on average.  Of those, in microseconds (rows, groups, N x K):
//   W4A16  16384, 64, 4096 x 1536   128x256: 209 * 64x256: 237   32x256: 321   64x128: 276   32x128: 330
//   W4A16  4096, 16, 4096 x 4096    128x256: 144 * 64x256: 157   32x256: 213   64x128: 177   32x128: 239
//   W4A16  768, 64, 3000 x 4096     128x256: 133   64x256: 104   32x256: 98 *  64x128: 115   32x128: 129
//   W4A16  1000, 128, 1536 x 2048   128x256: 72    64x256: 55    32x256: 50 *  64x128: 59    32x128: 54
//   W4A16  2000, 4, 700 x 1024      128x256: 21.5  64x256: 13.9  32x256: 10.7  64x128: 10.8* 32x128: 12.2
//   W4A16  100, 8, 4096 x 4096      128x256: 52    64x256: 37    32x256: 34    64x128: 26.8  32x128: 26.4 *
//   W4A4   32768, 64, 4096 x 2048   256x256: 240 * 128x256: 275  128x128: 352  64x128: 341
//   W4A4   3000, 64, 3000 x 4096    256x256: 106   128x256: 93 * 128x128: 109  64x128: 99
//   W4A4   500, 1, 4096 x 4096      256x256: 31.2  128x256: 20.0 128x128: 15.0 64x128: 12.4 *
//   W4A4   300, 8, 4096 x 4096      256x256: 30.6  128x256: 24.3 128x128: 20.7 64x128: 24.5 *
// (W4A4 in tiles of 32 rows was never faster than in 64; W4A16 in 256 x 256, or in 128 x 256 with eight waves of half the
// rows, 12 to 22 % slower: waves of 128 rows read fewer bytes from LDS an instruction, and two workgroups of four waves
// share a CU.)
constexpr int kGroupShapes[2] = {5, 4};
constexpr TileCost kGroupCost[2][5] = {
    {{128, 256, 4, 2, 9.65, 5.06, 9.58},
     {64, 256, 4, 2, 8.76, 3.46, 5.39},
     {32, 256, 4, 2, 2.21, 4.06, 5.34},
     {64, 128, 4, 2, 3.69, 2.37, 3.91},
     {32, 128, 2, 4, 1.21, 2.66, 6.41}},
    {{256, 256, 8, 1, 8.05, 2.39, 3.23},
     {128, 256, 8, 1, 5.46, 2.21, 2.21},
     {128, 128, 8, 1, 3.07, 2.10, 2.10},
     {64, 128, 4, 2, 3.51, 1.36, 2.02}},
};
constexpr double kGroupTail[2] = {0.24, 0.51};  // of a round, where there is more than one: the last is not full

// Most tiles of `bm` rows that `rows` rows in `groups` groups can take: a last one that is not full per group with rows.
inline int64_t group_tiles(int64_t rows, int64_t groups, int bm) {
    return rows / bm + (groups < rows ? groups : rows);
}

// The cheapest shape for groups of about the same size, of which only the sum is known here; -1 when no launch holds
// its tiles.  A group's last tile is half full on average.
inline int plan_grouped(int64_t rows, int64_t groups, int64_t N, int64_t K, bool a_mx, int num_cus) {
    const int64_t windows = (K + kPlanWindow - 1) / kPlanWindow;
    int best = -1;
    double cost = 1e30;
    for (int cfg = 0; cfg < kGroupShapes[a_mx ? 1 : 0]; cfg++) {
        const TileCost &t = kGroupCost[a_mx ? 1 : 0][cfg];
        const int64_t tn = (N + t.bn - 1) / t.bn;
        if ((uint64_t)tile_grid(group_tiles(rows, groups, t.bm) * tn) * 64 * t.waves > kMaxGridThreads) continue;
        const double used = (double)(groups < rows ? groups : rows);
        double tm = (double)rows / t.bm + used / 2;
        if (tm < used) tm = used;
        const double tiles = tm * (double)tn, slots = (double)num_cus * t.per_cu;
        const double rounds = tiles <= slots ? 1.0 : tiles / slots + kGroupTail[a_mx ? 1 : 0];
        const double us = tiles <= num_cus ? t.start + windows * t.window : rounds * (t.start + windows * t.window_full);
        if (us < cost) {
            cost = us;
            best = cfg;
        }
    }
    return best;
}

// Whether a grouped product with MXFP4 activations loads W past the caches.  Streamed, W does not drive out the lines of scale
// bytes, of which eight windows share one; but a row tile then finds nothing of W that another has loaded.  So where the L2s do
// not hold W anyway, or where most groups are one row tile.  Microseconds streamed and not (rows, groups, N x K; the pick marked):
//   768, 1, 3000 x 4096      22.7, 17.1 *     32768, 1, 4096 x 2048    197, 184 *      24000, 16, 700 x 1024   35.3, 33.1 *
//   1500, 4, 3000 x 4096     25.7, 23.3 *     16384, 8, 4096 x 2048    114, 111 *      6000, 2, 4096 x 8192    128, 123 *
//   256, 8, 4096 x 2048      14.0 *, 14.8     768, 64, 3000 x 4096     75.1 *, 79.6    200, 128, 4096 x 8192   213 *, 240
//   4096, 64, 4096 x 2048    86.4 *, 91.0     32768, 64, 4096 x 2048   252 *, 262      24000, 128, 1536 x 2048 96.2 *, 99.6
// It does not fit everywhere: 1500, 32, 3000 x 4096 59.8 *, 54.7; 1500, 16, the same 50.6 *, 47.3; 256, 1, 4096 x 2048 8.2, 8.8 *;
// 200, 2, 4096 x 8192 22.9, 24.0 *.
// (W4A16 never streams: its steps take a quarter of a line, and gate and up of 96 tokens took 166 instead of 100.)
inline bool grouped_streams(int64_t rows, int64_t groups, int64_t N, int64_t K) {
    return rows <= 32 * groups || groups * N * (K / 2) >= (int64_t)48 << 20;
}

}  // namespace nvfp4
