"""Low-rank adapters of many requests beside an MXFP4 projection, on the GPU against the plain float64 form."""
import pytest
import torch

import mx_shapes
from gpu_util import DEV, padded

pytestmark = pytest.mark.gpu
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def case(nv, seed, m, n, k, rank, count):
    g = gen(seed)
    a = randn(g, m, k).to(torch.bfloat16)
    w = nv.mx_quantize(randn(g, n, k) * 0.05)
    down = (randn(g, count, rank, k) * k ** -0.5).to(torch.bfloat16)
    up = (randn(g, count, n, rank) * 0.3).to(torch.bfloat16)
    scales = torch.rand(count, generator=g, device=DEV) + 0.5
    index = torch.randint(-1, count + 1, (m,), generator=g, device=DEV).to(torch.int32)  # none at both ends
    return a, w, down, up, scales, index


def expected(nv, a, w, down, up, scales, index, a_q=None):
    """(float64 C, bound on the error before its rounding)."""
    x, wd = a.double(), nv.mx_dequantize(w, torch.float32).double()
    main = x if a_q is None else nv.mx_dequantize(a_q, torch.float32).double()
    k, rank = w.shape[1], down.shape[1]
    # fp32 sums of products: a partial sum is at most the sum of the magnitudes and is rounded at most once per eight
    # products, and 16 more times in the joins of waves and slices
    steps = (k / 8 + 16) * 2.0 ** -24
    mag = main.abs() @ wd.abs().t()
    y, err = main @ wd.t(), steps * mag
    for j in torch.unique(index).tolist():
        if not 0 <= j < down.shape[0]:
            continue
        rows = (index == j).nonzero().flatten()
        s = 1.0 if scales is None else float(scales[j])
        v, u, xr = down[j].double(), up[j].double(), x[rows]
        t, dt = s * (xr @ v.t()), s * steps * (xr.abs() @ v.abs().t())
        dt = dt + 2.0 ** -23 * t.abs()  # the scale
        y[rows] += t @ u.t()
        # the up product, at worst: for few rows a rounding for each product and each sum of its own; for many it goes on the
        # product's sums, three planes of T one after the other, with a rounding per eight ranks of each
        tu = (t.abs() + dt) @ u.abs().t()
        err[rows] += dt @ u.abs().t() + (2 * rank + 8) * 2.0 ** -24 * tu + (3 * rank / 8 + 8) * 2.0 ** -24 * (mag[rows] + tu)
    return y, err + 2.0 ** -23 * y.abs()


def check(got, want, err, dt):
    info = torch.finfo(dt)
    diff = (got.double() - want).abs()
    assert bool((diff <= err * (1 + info.eps) + want.abs() * info.eps / 2 + info.tiny).all()), float((diff - err).max())


@pytest.mark.parametrize("act", ["bf16", "mx"])
@pytest.mark.parametrize("m, n, k, rank, count", [(1, 1, 32, 8, 1), (1, 4096, 512, 16, 5), (2, 100, 96, 24, 3), (5, 77, 1056, 40, 2), (8, 16, 128, 256, 9),
                                                  (13, 4200, 544, 8, 30), (16, 8300, 1024, 64, 16), (16, 50, 4128, 16, 1), (17, 33, 160, 32, 4), (48, 258, 2080, 16, 64),
                                                  (64, 128, 64, 72, 7), (65, 130, 96, 8, 2), (130, 64, 512, 24, 100), (200, 300, 1056, 128, 3), (700, 96, 640, 48, 40)])
def test_adapters(nv, m, n, k, rank, count, act):
    print(m, n, k, rank, count, act, flush=True)
    a, w, down, up, scales, index = case(nv, m + k, m, n, k, rank, count)
    a_q = nv.mx_quantize(a) if act == "mx" else None
    want, err = expected(nv, a, w, down, up, scales, index, a_q)
    for dt in TDT.values():
        check(nv.mx_gemm_adapters(a, w, down, up, index, scales=scales, a_q=a_q, dtype=dt), want, err, dt)
    want, err = expected(nv, a, w, down, up, None, index, a_q)
    buf = torch.full((m, n + 3), 7.0, device=DEV)
    nv.mx_gemm_adapters(padded(a, 8), w, down, up, index, a_q=a_q, out=buf[:, :n])
    check(buf[:, :n], want, err, torch.float32)
    assert bool((buf[:, n:] == 7).all())


@pytest.mark.parametrize("shape, act, tile, splits", mx_shapes.PRODUCTS)
def test_every_tile_shape(nv, shape, act, tile, splits):
    m, n, k = shape
    print(shape, act, tile, splits, flush=True)
    a, w, down, up, scales, index = case(nv, m, m, n, k, 24, 5)
    index[:m // 2] = 3  # a long request, then mixed rows
    a_q = nv.mx_quantize(a) if act == "mx" else None
    want, err = expected(nv, a, w, down, up, scales, index, a_q)
    for dt in TDT.values():
        check(nv.mx_gemm_adapters(a, w, down, up, index, scales=scales, a_q=a_q, dtype=dt), want, err, dt)
    # unsplit, with a workspace for T alone
    least = nv.lib.mxfp4_adapters_workspace_size(m, n, 32, 5, 24, act == "mx")
    ws = torch.empty(least, dtype=torch.uint8, device=DEV)
    check(nv.mx_gemm_adapters(a, w, down, up, index, scales=scales, a_q=a_q, workspace=ws), want, err, torch.float32)


@pytest.mark.parametrize("m", [1, 9, 16, 17, 100, 300])
@pytest.mark.parametrize("act", ["bf16", "mx"])
def test_rows_without_an_adapter_are_the_products_own(nv, m, act):
    a, w, down, up, scales, index = case(nv, m, m, 272, 544, 16, 4)
    a_q = nv.mx_quantize(a) if act == "mx" else None
    plain = nv.mx_gemm(a if a_q is None else a_q, w)
    got = nv.mx_gemm_adapters(a, w, down, up, index, scales=scales, a_q=a_q)
    none = (index < 0) | (index >= 4)
    assert torch.equal(got[none], plain[none])
    index[:] = torch.tensor([-1, 4, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV).repeat((m + 3) // 4)[:m]
    assert torch.equal(nv.mx_gemm_adapters(a, w, down, up, index, a_q=a_q), plain)
    assert torch.equal(nv.mx_gemm_adapters(a, w, down[:0], up[:0], index, a_q=a_q), plain)


@pytest.mark.parametrize("m", [6, 16, 40, 300])
def test_what_an_adapter_holds_stays_with_its_rows(nv, m):
    a, w, down, up, scales, index = case(nv, m, m, 272, 544, 16, 4)
    index[:] = torch.arange(m, device=DEV) % 4
    clean = nv.mx_gemm_adapters(a, w, down, up, index, scales=scales)
    mine, others = index == 2, index != 2
    for what in ("down", "up", "scales"):
        d, u, s = down.clone(), up.clone(), scales.clone()
        if what == "down":
            d[2, 5, 40] = float("nan")
        elif what == "up":
            u[2, :, 3] = float("inf")
        else:
            s[2] = float("inf")
        got = nv.mx_gemm_adapters(a, w, d, u, index, scales=s)
        assert torch.equal(got[others], clean[others])
        assert bool((~got[mine].isfinite()).any(1).all())
    # a row of A with a NaN or an infinity
    x = a.clone()
    x[1, 7], x[m - 1, 0] = float("nan"), float("inf")
    got = nv.mx_gemm_adapters(x, w, down, up, index, scales=scales)
    keep = [r for r in range(m) if r not in (1, m - 1)]
    assert torch.equal(got[keep], clean[keep]) and bool((~got[[1, m - 1]].isfinite()).all())


def test_large_and_small_values_of_t_keep_fp32s_bits(nv):
    # T = 2^100 + 2^80 + 2^77 needs three planes; U takes it apart again
    m, n, k, rank = 40, 64, 32, 8
    a = torch.zeros((m, k), dtype=torch.bfloat16, device=DEV)
    a[:, 0], a[:, 1], a[:, 2] = 2.0 ** 50, 2.0 ** 30, 2.0 ** 27
    w = nv.mx_quantize(torch.zeros((n, k), device=DEV))
    down = torch.zeros((1, rank, k), dtype=torch.bfloat16, device=DEV)
    down[0, 0, :3] = 2.0 ** 50
    down[0, 1, 0] = 2.0 ** 50
    up = torch.zeros((1, n, rank), dtype=torch.bfloat16, device=DEV)
    up[0, :, 0], up[0, :, 1] = 1, -1
    index = torch.zeros(m, dtype=torch.int32, device=DEV)
    for rows in (1, 16, m):
        y = nv.mx_gemm_adapters(a[:rows], w, down, up, index[:rows])
        assert bool((y == 2.0 ** 80 + 2.0 ** 77).all())


def test_empty_sides(nv):
    a, w, down, up, scales, index = case(nv, 1, 20, 64, 96, 8, 3)
    assert nv.mx_gemm_adapters(a[:0], w, down, up, index[:0]).shape == (0, 64)
    empty = nv.MXFP4Tensor.empty(64, 0, DEV)
    y = nv.mx_gemm_adapters(a[:, :0], empty, down[:, :, :0].contiguous(), up, index)
    assert y.shape == (20, 64) and bool((y == 0).all())
