"""The MXFP4 products' buffer loads on the CPU: every address that their offsets form, for every tile shape,
with whole tiles and with any number of rows missing, against the rows that there are.  A load that must not
happen has to be refused whether or not the scalar offset counts in the range check."""
import os
import re
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_gemm_nvfp4_amd", "csrc")

WALK = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "mx_bounds.h"
using namespace nvfp4::bounds;
typedef long long ll;

static ll loads, refused;
// One 16-byte load; `want` is its byte behind the operand's first row, or -1 when it must not happen.
static void load(ll base, ll bytes, ll voff, ll soff, ll want, ll extent) {
    loads++;
    const ll at = want < 0 ? voff : voff + 15;                                // a refused load is refused from its first byte on
    const bool lone = at >= bytes;                                            // the range check leaves the scalar offset out,
    const bool counted = (unsigned)at >= (unsigned)bytes - (unsigned)soff;    // or counts it
    if (want < 0) {
        refused++;
        if (!counted || !lone) { printf("not refused: bytes %lld voff %lld soff %lld\n", bytes, voff, soff); exit(1); }
    } else if (counted || lone || base + voff + soff != want || want + 16 > extent) {
        printf("wrong: bytes %lld voff %lld soff %lld want %lld\n", bytes, voff, soff, want);
        exit(1);
    }
}

// One operand of a tile: `per` units of 1 KiB per wave, rows of `rowb` bytes a step.
static void operand(int nw, int per, int rowb, int have, int steps, int nst, ll row_bytes, ll row_len) {
    const int pieces = rowb / 16, rpu = 64 / pieces;
    const ll extent = (have - 1) * row_bytes + row_len;
    for (int s = 0; s < steps + nst; s = s == 1 && steps > 6 ? steps - 3 : s + 1)
        for (int i = 0; i < per; i++) {
            const Part part = rows_part(i * nw * rpu, nw * rpu, have, (int)row_bytes, (int)row_len);
            for (int wave = 0; wave < nw; wave++)
                for (int lane = 0; lane < 64; lane += 1) {
                    const int r = wave * rpu + lane / pieces, at = lane % pieces * 16;  // (a swizzle only permutes `at`)
                    const int row = i * nw * rpu + r;
                    const ll col = (ll)s * rowb + at;
                    load(part.base, part.bytes, lane_off((uint32_t)(r * row_bytes), s * rowb, at, (int)row_len),
                         part_soff((uint32_t)(s * rowb), part.bytes),
                         row < have && col < row_len ? row * row_bytes + col : -1, extent);
                }
        }
}

// The codes of up to 16 rt rows as the form for few rows reads them.
static void few_rows(int rt, int rows, ll k, int waves) {
    const int full = (int)(k / 512), rb = (int)(k / 2);
    for (int g = 0; g < full + 2 * waves; g = g == 2 && full > 8 ? full - 2 : g + 1) {
        const uint32_t bytes = g < full ? (uint32_t)(rows * rb) : 0u, soff = part_soff((uint32_t)g * 256, bytes);
        for (int t = 0; t < rt; t++)
            for (int lane = 0; lane < 64; lane++)
                for (int i = 0; i < 4; i++) {
                    const int row = 16 * t + lane % 16 < rows ? 16 * t + lane % 16 : rows - 1, lg = lane / 16;
                    load(0, bytes, (uint32_t)(row * rb + lg * 16) + i * 64, soff,
                         g < full ? (ll)row * rb + g * 256 + i * 64 + lg * 16 : -1, (ll)rows * rb);
                }
    }
}

int main(int, char **v) {
    const int bm = atoi(v[1]), bn = atoi(v[2]), nw = atoi(v[3]), mx = atoi(v[4]), nst = atoi(v[5]);
    const int a_rowb = 128, bk = mx ? 256 : 64, w_rowb = bk / 2;
    for (ll k : {32ll, 96ll, 512ll, 544ll, 4128ll, 1ll << 22})
        for (ll pad : {0ll, 8ll, (1ll << 22) - k}) {
            const ll alen = mx ? k / 2 : 2 * k, arb = mx ? alen : 2 * (k + pad);
            const int steps = (int)((k + bk - 1) / bk);
            for (int have = 1; have <= bm; have += have < 3 || have > bm - 3 ? 1 : bm / 8 - 1)
                operand(nw, bm * a_rowb / 1024 / nw, a_rowb, have, steps, nst, arb, alen);
            for (int have = 1; have <= bn; have += have < 3 || have > bn - 3 ? 1 : bn / 8 - 1)
                operand(nw, bn * w_rowb / 1024 / nw, w_rowb, have, steps, nst, k / 2, k / 2);
        }
    for (int rt = 1; rt <= 3; rt++)
        for (int rows = 1; rows <= 16 * rt; rows++)
            for (ll k : {32ll, 512ll, 544ll, 6176ll, 1ll << 22}) few_rows(rt, rows, k, 4);
    printf("%lld loads, %lld of them refused\n", loads, refused);
    return refused > 0 ? 0 : 1;
}
"""


def tile_shapes():
    text = open(os.path.join(CSRC, "mx_gemm.hip")).read()
    found = re.findall(r"launch_tile_t<MxTile<(\d+), (\d+), (\d+), (\d+), (true|false), (\d+)>", text)
    return [(int(bm), int(bn), int(wm) * int(wn), int(mx == "true"), int(nst)) for bm, bn, wm, wn, mx, nst in found]


@pytest.fixture(scope="module")
def walker(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx_bounds")
    src, exe = d / "walk.cpp", d / "walk"
    src.write_text(WALK)
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    return str(exe)


def test_ten_tile_shapes_are_known():
    shapes = tile_shapes()
    assert len(shapes) == 10 and len(set(shapes)) == 10


@pytest.mark.parametrize("shape", tile_shapes(), ids=lambda s: "x".join(map(str, s)))
def test_loads_stay_within_their_rows(walker, shape):
    r = subprocess.run([walker, *map(str, shape)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
