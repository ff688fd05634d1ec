"""The plan of the MXFP4 products (tile shape and K slices), asked on the CPU."""
import ctypes
import os
import re
import subprocess

import pytest

import mx_shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_gemm_nvfp4_amd", "csrc")
CUS = 256

ASK = """
#include "mx_plan.h"
using namespace nvfp4;
extern "C" int shapes() { return kTileShapes; }
extern "C" int max_splits() { return kMaxSplits; }
extern "C" void shape(int mx, int cfg, int *bm, int *bn) { *bm = kTileCost[mx][cfg].bm; *bn = kTileCost[mx][cfg].bn; }
extern "C" int waves(int mx, int cfg) { return kTileCost[mx][cfg].waves; }
extern "C" void plan(int64_t m, int64_t n, int64_t k, int mx, int cus, uint64_t have, int *out) {
    const MxPlan p = plan_mx_within(m, n, k, mx, cus, have);
    out[0] = p.cfg; out[1] = p.splits; out[2] = p.slice_windows;
}
extern "C" void plan_unsplit(int64_t m, int64_t n, int64_t k, int mx, int cus, int *out) {
    const MxPlan p = plan_mx(m, n, k, mx, cus, 1);
    out[0] = p.cfg; out[1] = p.splits; out[2] = p.slice_windows;
}
"""
ALL = (1 << 64) - 1


@pytest.fixture(scope="module")
def ask(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx_plan")
    src, so = d / "ask.cpp", d / "ask.so"
    src.write_text(ASK)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    i64 = ctypes.c_int64
    lib.plan.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.c_uint64, ctypes.POINTER(ctypes.c_int)]
    lib.plan_unsplit.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]

    class Ask:
        shapes, max_splits = lib.shapes(), lib.max_splits()

        @staticmethod
        def tile(mx, cfg):
            bm, bn = ctypes.c_int(), ctypes.c_int()
            lib.shape(mx, cfg, ctypes.byref(bm), ctypes.byref(bn))
            return bm.value, bn.value

        @staticmethod
        def waves(mx, cfg):
            return lib.waves(mx, cfg)

        @staticmethod
        def plan(m, n, k, mx, have=ALL):
            out = (ctypes.c_int * 3)()
            lib.plan(m, n, k, mx, CUS, have, out)
            return tuple(out)

        @staticmethod
        def unsplit(m, n, k, mx):
            out = (ctypes.c_int * 3)()
            lib.plan_unsplit(m, n, k, mx, CUS, out)
            return tuple(out)
    return Ask


@pytest.mark.parametrize("mx", [0, 1])
def test_without_its_workspace_a_product_takes_the_shape_that_is_cheapest_in_one_piece(ask, mx):
    seen = set()
    for m, n, k in [(512, 4096, 12288), (128, 4096, 4096), (17, 288, 1088), (130, 8288, 10336), (65, 5392, 7744),
                    (193, 16416, 11360), (17, 280, 2624), (512, 8192, 1 << 22)]:
        cfg, splits, windows = ask.plan(m, n, k, mx)
        assert 1 <= splits <= ask.max_splits and (splits - 1) * windows < -(-k // 512) <= splits * windows
        need = splits * m * n * 4 if splits > 1 else 0
        assert ask.plan(m, n, k, mx, need) == (cfg, splits, windows)
        one = ask.unsplit(m, n, k, mx)
        assert one[1:] == (1, -(-k // 512))
        for have in {0, need - 1, need // 2} if need else {0}:
            assert ask.plan(m, n, k, mx, have) == one
        seen.add((cfg != one[0], splits > 1))
    assert (True, True) in seen  # the shapes of the two forms do differ somewhere


def test_the_products_of_the_gpu_tests_reach_every_shape(ask):
    reached = set()
    for (m, n, k), act, tile, splits in mx_shapes.PRODUCTS:
        mx = int(act == "mx")
        cfg, s, _ = ask.plan(m, n, k, mx)
        assert (ask.tile(mx, cfg), s) == (tile, splits), (m, n, k, act, ask.tile(mx, cfg), s)
        assert m % tile[0] and n % tile[1] and k % (256 if mx else 64) and n > tile[1] and n % 8 == 0
        reached.add((mx, cfg, s > 1))
    assert reached == {(mx, cfg, split) for mx in (0, 1) for cfg in range(ask.shapes) for split in (False, True)}


def test_the_kernels_are_the_shapes_of_the_table(ask):
    text = open(os.path.join(CSRC, "mx_gemm.hip")).read()
    for mx, word in ((0, "false"), (1, "true")):
        found = re.findall(r"launch_tile_t<MxTile<(\d+), (\d+), (\d+), (\d+), %s, \d+>" % word, text)
        assert [(int(a), int(b), int(c) * int(d)) for a, b, c, d in found] == \
            [(*ask.tile(mx, c), ask.waves(mx, c)) for c in range(ask.shapes)]


@pytest.mark.parametrize("mx", [0, 1])
def test_one_launch_holds_the_tiles(ask, mx):
    most = (1 << 31) - (1 << 11)
    assert ask.plan(1 << 31, 1 << 31, 32, mx)[0] < 0
    for m, n in ((1 << 28, 3), (1 << 30, 1), ((1 << 30) + 100, 1), (most, 1), (17, most), (1 << 20, 1 << 11)):
        cfg, _, _ = ask.plan(m, n, 32, mx)
        bm, bn = ask.tile(mx, cfg)
        tiles = -(-m // bm) * -(-n // bn)
        assert -(-tiles // 8) * 8 * 64 * ask.waves(mx, cfg) < 1 << 32, (m, n)


def test_products_of_more_tiles_than_a_launch_holds_are_refused():
    import bit_gemm_nvfp4_amd as nv
    from bit_gemm_nvfp4_amd.mx import CMXTensor
    fake, most = 0x10000, (1 << 31) - (1 << 11)  # 16-byte aligned, never dereferenced

    def call(m, n):
        a, w = CMXTensor(fake, fake, m, 32), CMXTensor(fake, fake, n, 32)
        return nv.lib.mxfp4_gemm(None, ctypes.byref(a), m, 0, ctypes.byref(w), ctypes.c_void_p(fake), 0, n, None, 1 << 40, None)
    assert call(most + 1, 1) == 2 and call(17, most + 1) == 2
