"""Where the grouped products with MXFP4 activations load W past the caches, on the CPU."""
import ctypes
import os
import random
import subprocess

import pytest

import mx_stream_shapes

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemm_nvfp4_amd", "csrc")


@pytest.fixture(scope="module")
def streams(tmp_path_factory):
    d = tmp_path_factory.mktemp("mx_group_stream")
    src, so = d / "ask.cpp", d / "ask.so"
    src.write_text('#include "mx_plan.h"\nextern "C" int streams(int64_t r, int64_t g, int64_t n, int64_t k)'
                   ' { return nvfp4::grouped_streams(r, g, n, k); }\n'
                   'extern "C" int tile(int64_t r, int64_t g, int64_t n, int64_t k)'
                   ' { auto &t = nvfp4::kGroupCost[1][nvfp4::plan_grouped(r, g, n, k, true, 256)]; return t.bm * 1000 + t.bn; }\n')
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    lib.streams.argtypes = lib.tile.argtypes = [ctypes.c_int64] * 4

    def streams(*a):
        return bool(lib.streams(*a))
    streams.tile = lambda *a: divmod(lib.tile(*a), 1000)
    return streams


# measured: a W that several row tiles share and the caches hold was up to a third slower when it passed them by
@pytest.mark.parametrize("rows, groups, n, k", [(768, 1, 3000, 4096), (1500, 4, 3000, 4096), (16384, 8, 4096, 2048), (32768, 1, 4096, 2048),
                                                (24000, 16, 700, 1024), (6000, 2, 4096, 8192), (6000, 16, 1536, 2048)])
def test_a_shared_w_stays_in_the_caches(streams, rows, groups, n, k):
    assert not streams(rows, groups, n, k)


@pytest.mark.parametrize("rows, groups, n, k", [(256, 64, 4096, 2048), (768, 64, 3000, 4096), (256, 8, 4096, 2048), (200, 128, 4096, 8192),
                                                (32768, 64, 4096, 2048), (24000, 128, 1536, 2048), (16384, 64, 3000, 4096)])
def test_a_w_read_once_or_larger_than_the_caches_passes_them(streams, rows, groups, n, k):
    assert streams(rows, groups, n, k)


def test_the_largest_sizes_do_not_wrap(streams):
    assert streams(1 << 24, 512, 1 << 24, 1 << 20) and not streams(1 << 24, 1, 1, 32)


def test_shapes_of_the_gpu_tests(streams):
    for (sizes, n, k), tile in mx_stream_shapes.STREAMED:
        args = sum(sizes), len(sizes), n, k
        assert streams(*args) and streams.tile(*args) == tile, args


def test_no_streamed_product_takes_the_shape_that_has_no_such_kernel(streams):
    rng = random.Random(1)
    for _ in range(100000):
        args = rng.randint(1, 40000), rng.randint(1, 512), rng.randint(2, 9000), 32 * rng.randint(1, 600)
        assert not streams(*args) or streams.tile(*args) != (128, 128), args
