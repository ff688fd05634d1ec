"""Lanes of one wave that hand values to each other through LDS: between a lane's store and another lane's load of the same
word, and between a load and another lane's store over it, stands a fence, on every way through the compiled code.  Without
one their order is the compiler's to choose."""
import re

import pytest

import gfx_ir

WAVES, MAX_GROUPS = 16, 512
COUNTS = WAVES * MAX_GROUPS * 4  # bytes of the counts per wave and group, the first array of the kernels' LDS


@pytest.fixture(scope="module")
def route(tmp_path_factory):
    return gfx_ir.functions(gfx_ir.compiled(tmp_path_factory.mktemp("mx_route_ir"), "mx_route.hip"))


def counts(kinds):
    return lambda kind, ty, off: kind in kinds and off is not None and off < COUNTS


def kernels(found, name):
    return {n: gfx_ir.Lds(f) for n, f in found.items() if re.search(r"\d" + name + r"(I|E)", n)}


@pytest.mark.parametrize("name, many", [("k_mx_place", 1), ("k_mx_count", 1), ("k_mx_route", 8)])
def test_counts_of_a_wave(route, name, many):
    found = kernels(route, name)
    assert len(found) == many
    for kernel, f in found.items():
        seen = [k for body, _ in f.blocks.values() for k, ty, off in f.steps(body) if counts("LSX")(k, ty, off)]
        assert "S" in seen and "L" in seen, kernel
        # (within a block the same lanes do both, each on words of its own)
        for first, then in (("S", "LX"), ("L", "SX"), ("X", "LS")):
            assert not f.unordered(counts(first), counts(then), same_block=False), (kernel, first, then)


CODE = """
  br label %2

2:                                                ; preds = %5, %0
  %3 = getelementptr inbounds i32, ptr addrspace(3) @lds, i32 %1
  %4 = load i32, ptr addrspace(3) %3, align 4
  br i1 %first, label %5, label %7

5:                                                ; preds = %2
  store i32 %6, ptr addrspace(3) %3, align 4
  fence syncscope("wavefront") release
  br i1 %again, label %2, label %7

7:                                                ; preds = %5, %2
  ret void
"""


def test_the_walk_finds_the_ways_without_a_fence():
    f = gfx_ir.Lds(CODE.splitlines())
    assert len(f.unordered(counts("L"), counts("S"), same_block=False)) == 1
    assert not f.unordered(counts("S"), counts("L"), same_block=False)
    bare = gfx_ir.Lds([ln for ln in CODE.splitlines() if "fence" not in ln])
    assert len(bare.unordered(counts("S"), counts("L"), same_block=False)) == 1
    assert f.offset("getelementptr inbounds nuw (i8, ptr addrspace(3) @lds, i32 32768), i32 %9") == 32768


@pytest.fixture(scope="module")
def compiled(tmp_path_factory):
    done, tmp = {}, tmp_path_factory.mktemp("mx_wave_ir")

    def get(source):
        if source not in done:
            done[source] = gfx_ir.functions(gfx_ir.compiled(tmp, source))
        return done[source]
    return get


# Sums on their way to C: each wave writes rows of its own part of LDS, a value a lane, and reads them back as whole pieces.
@pytest.mark.parametrize("source, name, many", [("mx_grouped.hip", "k_mx_grouped", 60), ("mx_gemm.hip", "k_mx_tile", 30),
                                                ("mx_gemm.hip", "k_adapter_tile", 30)])
def test_sums_on_their_way_to_c(compiled, source, name, many):
    found = kernels(compiled(source), name)
    assert len(found) == many
    value, piece = lambda kind, ty, off: (kind, ty) == ("S", "float"), lambda kind, ty, off: (kind, ty) == ("L", "<4 x float>")
    for kernel, f in found.items():
        assert sum(value(*s) for body, _ in f.blocks.values() for s in f.steps(body)) >= 16, kernel
        assert not f.unordered(value, piece, same_block=True), kernel
        assert not f.unordered(piece, value, same_block=True), kernel


def test_sums_of_a_token_in_the_layer_for_few_tokens(compiled):
    # a token's sums are added to by whichever lanes hold it in the expert at hand
    found = kernels(compiled("mx_moe.hip"), "k_moe_down")
    assert len(found) == 4
    for kernel, f in found.items():
        store, load = lambda kind, ty, off: (kind, ty) == ("S", "<4 x float>"), lambda kind, ty, off: (kind, ty) == ("L", "<4 x float>")
        assert any(store(*s) for body, _ in f.blocks.values() for s in f.steps(body)), kernel
        assert not f.unordered(store, load, same_block=False), kernel
