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

// The cheapest of the shapes and of up to `max_splits` K slices.
inline MxPlan plan_mx(int64_t M, int64_t N, int64_t K, bool a_mx, int num_cus, int max_splits = kMaxSplits) {
    const int64_t windows = (K + kPlanWindow - 1) / kPlanWindow;
    MxPlan best{-1, 1, (int)windows};
    double cost = 1e30;
    for (int cfg = 0; cfg < kTileShapes; cfg++) {
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
inline MxPlan plan_mx_within(int64_t M, int64_t N, int64_t K, bool a_mx, int num_cus, uint64_t have) {
    const MxPlan p = plan_mx(M, N, K, a_mx, num_cus);
    return plan_ws_bytes(p, M, N) <= have ? p : plan_mx(M, N, K, a_mx, num_cus, 1);
}

}  // namespace nvfp4
