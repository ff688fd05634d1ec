"""The MXFP4 products on the GPU at the sizes that reach their tile shapes and limits."""
import pytest
import torch

import mx_ref
import mx_shapes
from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


def _random(nv, g, rows, cols):
    """Random codes and scale bytes, every block with its own, and the values they stand for in float64."""
    codes = torch.randint(0, 256, (rows, cols // 2), generator=g, dtype=torch.uint8, device=DEV)
    scales = torch.randint(117, 130, (rows, cols // 32), generator=g, dtype=torch.uint8, device=DEV)
    table = torch.tensor([*mx_ref.E2M1, *-mx_ref.E2M1], dtype=torch.float64, device=DEV)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), dim=2).view(rows, cols // 32, 32)
    v *= torch.exp2(scales.double() - 127).unsqueeze(2)
    return nv.MXFP4Tensor(codes, scales), v.view(rows, cols)


@pytest.mark.parametrize("case", mx_shapes.PRODUCTS, ids=lambda c: "x".join(map(str, c[0])) + "-" + c[1])
def test_every_tile_shape(nv, case):
    (m, n, k), act, _, splits = case
    g = torch.Generator(device=DEV)
    g.manual_seed(m * n + k)
    w, wd = _random(nv, g, n, k)
    if act == "mx":
        a, ad = _random(nv, g, m, k)
    else:
        a = (torch.randn((m, k), generator=g, device=DEV) *
             torch.exp2(torch.randint(-6, 4, (m, k), generator=g, device=DEV).float())).to(torch.bfloat16)
        ad = a.double()
    ref, mag = ad @ wd.t(), ad.abs() @ wd.abs().t()
    bound = mx_ref.fp32_sum_bound(1, k) * mag

    def check(c):
        half = 2.0 ** -8 if c.dtype == torch.bfloat16 else 2.0 ** -24
        over = (c.double() - ref).abs() - bound - half * ref.abs() - 1e-38
        assert float(over.max()) <= 0, (int(over.argmax()) // n, int(over.argmax()) % n)
        return c
    ws = nv.mx_gemm_workspace(a, w)
    assert (ws is not None) == (splits > 1)
    f = check(nv.mx_gemm(a, w, workspace=ws))
    b = check(nv.mx_gemm(a, w, dtype=torch.bfloat16, workspace=ws))
    assert torch.equal(f.to(torch.bfloat16), b)
    # rows of C that allow no wide store, what lies around them left as it was
    buf = torch.full((m + 1, n + 3), 7.0, device=DEV)
    nv.mx_gemm(a, w, out=buf[:m, 1:n + 1], workspace=ws)
    assert torch.equal(buf[:m, 1:n + 1], f)
    buf[:m, 1:n + 1] = 7
    assert bool((buf == 7).all())
    if splits > 1:  # in one piece, the shape that is cheapest then
        check(nv.mx_gemm(a, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)))


def test_longest_rows_in_the_largest_tile(nv):
    # K and lda at their limit, in tiles of 256 rows: the last elements of a tile's last row are 2 GiB behind
    # its first
    m, n, k = 512, 8192, 1 << 22
    w = nv.MXFP4Tensor(torch.zeros((n, k // 2), dtype=torch.uint8, device=DEV),
                       torch.full((n, k // 32), 127, dtype=torch.uint8, device=DEV))
    w.codes[5, k // 2 - 1] = 0x42   # 1 and 2 as the last two elements
    w.codes[n - 1, k // 2 - 1] = 0x24
    a = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    a[:, k - 2] = torch.arange(m, device=DEV) % 128 + 1
    a[:, k - 1] = torch.arange(m, device=DEV) % 64 + 1
    c = nv.mx_gemm(a, w)
    want = torch.zeros((m, n), device=DEV)
    x, y = a[:, k - 2].float(), a[:, k - 1].float()  # the sums need more bits than bf16 has
    want[:, 5] = x + 2 * y
    want[:, n - 1] = 2 * x + y
    assert torch.equal(c, want)


def test_more_rows_than_small_tiles_fit_in_a_launch(nv):
    m = (1 << 30) + 100  # in tiles of 64 rows, more threads than one launch can have
    a = nv.MXFP4Tensor(torch.zeros((m, 16), dtype=torch.uint8, device=DEV),
                       torch.full((m, 1), 127, dtype=torch.uint8, device=DEV))
    w = nv.MXFP4Tensor(torch.full((1, 16), 0x22, dtype=torch.uint8, device=DEV),
                       torch.full((1, 1), 127, dtype=torch.uint8, device=DEV))
    rows = torch.tensor([0, 12345, 1 << 29, m - 101, m - 1], device=DEV)
    a.codes[rows] = 0x44
    c = nv.mx_gemm(a, w, dtype=torch.bfloat16)
    assert bool((c[rows] == 64).all()) and int((c != 0).sum()) == len(rows)


@pytest.mark.parametrize("m", [1, 6, 16, 40, 66])
@pytest.mark.parametrize("act", ["mx", "bf16"])
def test_smallest_and_largest_scales(nv, act, m):
    # one column of C per scale byte and pattern of codes; products and sums of a few of them, exact in fp32 down to its
    # subnormal numbers
    patterns = [[1], [2], [7], [1, 2, 7], [9, 10, 7], [3, 5, 11, 6]]
    n = 255 * len(patterns)
    codes = torch.zeros((n, 16), dtype=torch.uint8, device=DEV)
    for p, pat in enumerate(patterns):
        for j, c in enumerate(pat):
            codes[p::len(patterns), j] = c  # elements 0, 2, 4, ...
    scales = (torch.arange(n, device=DEV) // len(patterns)).to(torch.uint8).view(n, 1)
    w = nv.MXFP4Tensor(codes, scales)
    table = torch.tensor([*mx_ref.E2M1, *-mx_ref.E2M1], dtype=torch.float64, device=DEV)
    terms = table[codes.int()] * torch.exp2(scales.double() - 127)  # [n, 16] elements 0, 2, ...
    for e in (0, -20, 1, 60):
        a = torch.zeros((m, 32), dtype=torch.bfloat16, device=DEV)
        a[:, ::2] = 2.0 ** e
        c = nv.mx_gemm(nv.mx_quantize(a) if act == "mx" else a, w)
        if act == "bf16":  # W as bf16: values from 2^128 on are infinities
            big = terms.abs() >= 2.0 ** 128
            v = torch.where(big, torch.copysign(torch.full_like(terms, float("inf")), terms), terms)
        else:
            v = terms
        want = (v * 2.0 ** e).sum(dim=1)
        exact = (want.abs() / 2.0 ** -149 % 1 == 0) | ~torch.isfinite(want)  # a multiple of fp32's smallest step
        # the sums of the finite terms stay in fp32's range (-2^127 * 2 beside an infinity would be a NaN)
        inside = torch.where(v.isfinite(), v, torch.zeros_like(v)).abs().sum(dim=1) * 2.0 ** e < 2.0 ** 128
        keep = exact & inside
        got = c.double()
        ok = (got == want.float().double()) | (torch.isnan(got) & torch.isnan(want))
        assert bool(ok[:, keep].all()), (e, (~ok & keep).nonzero()[:4].tolist())
        assert int(keep.sum()) > n // 2
