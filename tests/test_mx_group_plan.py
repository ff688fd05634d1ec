"""Tile shapes and loads of the products grouped by rows, on the CPU."""
import ctypes
import os
import re
import subprocess

import pytest

import mx_group_shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_gemm_nvfp4_amd", "csrc")
CUS = 256

ASK = """
#include "mx_plan.h"
using namespace nvfp4;
extern "C" int shapes(int mx) { return kGroupShapes[mx]; }
extern "C" void shape(int mx, int cfg, int *bm, int *bn, int *waves) {
    const TileCost &t = kGroupCost[mx][cfg];
    *bm = t.bm; *bn = t.bn; *waves = t.waves;
}
extern "C" int plan(int64_t rows, int64_t groups, int64_t n, int64_t k, int mx, int cus) {
    return plan_grouped(rows, groups, n, k, mx, cus);
}
extern "C" int64_t most_tiles(int64_t rows, int64_t groups, int bm) { return group_tiles(rows, groups, bm); }
"""


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx_group_plan")
    src, so = d / "ask.cpp", d / "ask.so"
    src.write_text(ASK)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    i64 = ctypes.c_int64
    lib.plan.argtypes = [i64, i64, i64, i64, ctypes.c_int, ctypes.c_int]
    lib.most_tiles.argtypes, lib.most_tiles.restype = [i64, i64, ctypes.c_int], i64
    return lib


def shape(lib, mx, cfg):
    v = [ctypes.c_int() for _ in range(3)]
    lib.shape(mx, cfg, *[ctypes.byref(x) for x in v])
    return tuple(x.value for x in v)


def launched_shapes():
    """(bm, bn, waves, stages) of the launches, by activation kind, in the order of the plan's table."""
    text = open(os.path.join(CSRC, "mx_grouped.hip")).read()
    found = re.findall(r"launch_t<MxTile<(\d+), (\d+), (\d+), (\d+), (true|false), (\d+)>", text)
    out = {0: [], 1: []}
    for bm, bn, wm, wn, mx, nst in found:
        out[int(mx == "true")].append((int(bm), int(bn), int(wm) * int(wn), int(nst)))
    return out


def test_the_table_is_what_is_launched(ask):
    for mx, shapes in launched_shapes().items():
        assert len(shapes) == ask.shapes(mx)
        assert [s[:3] for s in shapes] == [shape(ask, mx, c) for c in range(ask.shapes(mx))]


def test_shapes_of_the_gpu_tests(ask):
    seen = set()
    for (sizes, n, k), act, tile in mx_group_shapes.GROUPED:
        cfg = ask.plan(sum(sizes), len(sizes), n, k, act == "mx", CUS)
        assert shape(ask, act == "mx", cfg)[:2] == tile, (sizes, n, k, act)
        seen.add((act, tile))
    assert len(seen) == ask.shapes(0) + ask.shapes(1)


def test_the_grid_holds_the_tiles_of_any_sizes(ask):
    import random
    rng = random.Random(3)
    for _ in range(2000):
        groups = rng.randint(1, 512)
        sizes = [rng.choice([0, 1, rng.randint(1, 40), rng.randint(1, 700)]) for _ in range(groups)]
        for bm in (32, 64, 128, 256):
            assert sum(-(-s // bm) for s in sizes) <= ask.most_tiles(sum(sizes), groups, bm)


def test_a_launch_that_no_shape_fits_is_not_planned(ask):
    for mx in (0, 1):
        assert ask.plan(1 << 24, 512, 1 << 24, 32, mx, CUS) == -1
        assert ask.plan(1 << 24, 512, 4096, 32, mx, CUS) >= 0


WALK = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "mx_bounds.h"
using namespace nvfp4::bounds;
typedef long long ll;

static ll loads, refused;
static void load(ll bytes, ll voff, ll soff, ll want) {
    loads++;
    const ll at = want < 0 ? voff : voff + 15;
    const bool lone = at >= bytes, counted = (unsigned)at >= (unsigned)bytes - (unsigned)soff;
    if (voff + soff > 0xFFFFFFFFll) { printf("offset wraps\n"); exit(1); }
    if (want < 0) {
        refused++;
        if (!counted || !lone) { printf("not refused: bytes %lld voff %lld soff %lld\n", bytes, voff, soff); exit(1); }
    } else if (counted || lone || voff + soff != want) {
        printf("wrong: bytes %lld voff %lld soff %lld want %lld\n", bytes, voff, soff, want);
        exit(1);
    }
}

// A lane whose row is `row` of a buffer of `have` rows (-1: none), at each step of the loop and the stages behind it.
static void lane(ll row, ll have, int rowb, int bk_steps, int nst, ll row_bytes, ll row_len) {
    const ll bytes = have ? (have - 1) * row_bytes + row_len : 0;
    for (int s = 0; s < bk_steps + nst; s = s == 1 && bk_steps > 6 ? bk_steps - 3 : s + 1)
        for (int at = 0; at < rowb; at += 16) {
            const ll col = (ll)s * rowb + at;
            const uint32_t off = step_off(row_off((int)row, (int)row_bytes, at), s * rowb, at, (int)row_len);
            load(bytes, off, part_soff((uint32_t)(s * rowb), (uint32_t)bytes),
                 row >= 0 && col < row_len ? row * row_bytes + col : -1);
        }
}

int main(int, char **v) {
    const int bm = atoi(v[1]), bn = atoi(v[2]), mx = atoi(v[3]), nst = atoi(v[4]);
    const int a_rowb = 128, bk = mx ? 256 : 64, w_rowb = bk / 2;
    for (ll k : {32ll, 96ll, 512ll, 544ll, 4128ll, 1ll << 20}) {
        const int steps = (int)((k + bk - 1) / bk);
        for (ll pad : {0ll, 8ll, (1ll << 20) - k}) {
            const ll alen = mx ? k / 2 : 2 * k, arb = mx ? alen : 2 * (k + pad);
            for (ll have : {1ll, 2ll, (ll)bm})  // the tile's own rows
                for (ll r = -1; r < have; r += r < 2 || r > have - 4 ? 1 : bm / 8 - 1) lane(r, have, a_rowb, steps, nst, arb, alen);
            const ll most = ((1ll << 31) - 1) / arb;  // picked from all of A
            for (ll have : {0ll, 1ll, most})
                for (ll r : {-1ll, 0ll, have / 2, have - 1})
                    if (r < have) lane(r, have, a_rowb, steps, nst, arb, alen);
        }
        const ll cols = ((1ll << 30) - 1) / (k / 2);  // gate and up rows of the largest group
        for (ll have : {1ll, (ll)bn, 2 * cols})
            for (ll r : {-1ll, 0ll, have / 2, have - 1}) lane(r, have, w_rowb, steps, nst, k / 2, k / 2);
    }
    // the adapters' first product: chunks of 256 or 512 bytes of rows of A (its tile's own or picked from all) and of V
    for (ll k : {32ll, 96ll, 544ll, 4128ll, 1ll << 21})
        for (int rowb : {256, 512})
            for (ll pad : {0ll, 8ll, (1ll << 21) - k}) {
                const ll row_bytes = 2 * (k + pad), row_len = 2 * k;
                const int steps = (int)((row_len + rowb - 1) / rowb);
                for (ll have : {1ll, 16ll, 64ll, ((1ll << 31) - 1) / row_bytes})
                    for (ll r : {-1ll, 0ll, have / 2, have - 1}) lane(r, have, rowb, steps, nst, row_bytes, row_len);
            }
    // T and U of a tile: 64 ranks at a time
    for (ll rank = 8; rank <= 256; rank += 8)
        for (ll have : {1ll, (ll)bm, (ll)bn})
            for (ll r : {-1ll, 0ll, have / 2, have - 1}) lane(r, have, 128, (int)((rank + 63) / 64), 1, 2 * rank, 2 * rank);
    printf("%lld loads, %lld of them refused\n", loads, refused);
    return refused > 0 ? 0 : 1;
}
"""


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx_group_bounds")
    src, exe = d / "walk.cpp", d / "walk"
    src.write_text(WALK)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return str(exe)


@pytest.mark.parametrize("mx, tile", [(mx, s) for mx, shapes in launched_shapes().items() for s in shapes])
def test_loads_stay_within_their_rows(walker, mx, tile):
    bm, bn, _, nst = tile
    r = subprocess.run([walker, str(bm), str(bn), str(mx), str(nst)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
