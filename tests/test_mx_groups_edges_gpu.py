"""Grouped products, router, weighted sum and expert layer at sizes and arguments that their other tests leave out."""
import numpy as np
import pytest
import torch

import mx_ref
import mx_stream_shapes
from gpu_util import DEV
from test_mx_groups_gpu import check, check_sort, expected, experts, offsets_of, operands, sum_bound

pytestmark = pytest.mark.gpu


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


def test_an_mxfp4_output_keeps_no_earlier_flags(nv):
    g = gen(1)
    x = randn(g, 40, 64)
    x[3, 5] = float("nan")
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = nv.mx_quantize(x, flags=flags)
    assert q.flags is flags and int(flags) == 1
    a, w = randn(g, 40, 96).to(torch.bfloat16), nv.mx_quantize(randn(g, 128, 96) * 0.1)
    nv.mx_grouped_gemm(a, w, torch.tensor([0, 40], dtype=torch.int32, device=DEV), swiglu=True, out=q)
    assert q.flags is None and bool(nv.mx_dequantize(q).isfinite().all())


# A workgroup of the router takes more than one round of 64 rows from 16385 rows on.
@pytest.mark.parametrize("t, e, k, dt", [(16385, 8, 2, torch.float32), (40000, 33, 3, torch.bfloat16), (33000, 300, 16, torch.float32)])
def test_route_of_many_rows(nv, t, e, k, dt):
    g = gen(t)
    logits = (randn(g, t, e) * 2).to(dt)
    logits[torch.rand((t, e), generator=g, device=DEV) < 0.1] = float("-inf")
    logits[16384:16386], logits[-1] = 0.5, float("-inf")
    logits[16000, 0] = float("nan")
    r = nv.mx_route(logits, k)
    lg = logits.double().cpu().numpy()
    ids, wts = mx_ref.route(lg, k, True)
    wts[16000] = np.nan
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    fin = np.where(np.isfinite(lg), lg, 0)
    tol = (2 * (fin.max(axis=1) - fin.min(axis=1)) + 40) * 2.0 ** -24  # as for fewer rows (test_route)
    got = r.weights.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(wts))
    assert (np.abs(np.nan_to_num(got) - np.nan_to_num(wts)) <= tol[:, None] * np.nan_to_num(wts) + 2.0 ** -126).all()
    check_sort(r, ids, e)


@pytest.mark.parametrize("zt, yt", [(torch.float32, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_combine_of_more_rows_than_a_grid_has(nv, zt, yt):
    t, k, p, cols = 65535 + 300, 2, 5000, 12
    g = gen(3)
    z = randn(g, p, cols).to(zt)
    places = torch.randint(-1, p, (t, k), generator=g, device=DEV).to(torch.int32)
    weights = torch.rand((t, k), generator=g, device=DEV)
    zd = torch.where((places >= 0).unsqueeze(2), z.double()[places.long().clamp(min=0)], 0.0)
    terms = zd * weights.double().unsqueeze(2)
    check(nv.mx_combine(z, places, weights, dtype=yt), terms.sum(1), 2 * k * 2.0 ** -24 * terms.abs().sum(1), yt)


# ------------------------------------------------------------------------------------------------
# the layer with quantized activations, against float64
# ------------------------------------------------------------------------------------------------
def on_grid(v, scale):
    """float64 v to the nearest E2M1 value times scale: ties to the even code, 6 beyond."""
    a = (v.abs() / scale).clamp(max=6)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v) * scale


def block_scales(v):
    """2^(floor(log2 max|v|) - 2) of each block of 32, for every element."""
    top = v.view(v.shape[0], -1, 32).abs().amax(2, keepdim=True)
    return torch.ldexp(torch.ones_like(top), torch.frexp(top)[1] - 3).expand(-1, -1, 32).reshape(v.shape)


def quantized(v, dv):
    """(v through MXFP4, how far the same may lie from it for values within dv of v)."""
    s = block_scales(v)
    q = on_grid(v, s)
    err = torch.maximum(on_grid(v + dv, s) - q, q - on_grid(v - dv, s))
    # a block whose maximum may pass a power of two may have the next scale; either grid is off by a quarter of a value, or of
    # the (larger) scale below one
    shaky = (block_scales(v.abs() + dv) != s) | (block_scales((v.abs() - dv).clamp(min=0)) != s)
    any_ = 2 * torch.maximum((v.abs() + dv) / 4, s / 2) + dv
    return q, torch.where(shaky, any_, err)


@pytest.mark.parametrize("logits_dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("quantize_acts", [True, False])
@pytest.mark.parametrize("t, e, k, h, i", [(7, 5, 2, 64, 96), (200, 6, 3, 160, 64), (1500, 40, 4, 96, 32)])
def test_layer_against_float64(nv, t, e, k, h, i, quantize_acts, logits_dt):
    x, logits, gu, dn = experts(nv, t + 1, t, e, h, i)
    logits = logits.to(logits_dt)
    y, got_ids, got_wts = nv.mx_experts(x, logits, gu, dn, k, quantize_acts=quantize_acts, dtype=torch.float32, routing=True)
    ids, wts = mx_ref.route(logits.double().cpu().numpy(), k, True)
    assert np.array_equal(got_ids.cpu().numpy(), ids)
    # (2 |d| + 40) 2^-24 for logits |d| apart, as in test_route, and these lie less than 40 apart
    assert np.abs(got_wts.double().cpu().numpy() - wts).max() <= 2.0 ** -17
    gud, dnd = nv.mx_dequantize(gu, torch.float32).double(), nv.mx_dequantize(dn, torch.float32).double()
    xd = x.double()
    if quantize_acts:
        xd = on_grid(xd, block_scales(xd))
    want, err = torch.zeros((t, h), dtype=torch.float64, device=DEV), torch.zeros((t, h), dtype=torch.float64, device=DEV)
    for j in range(e):
        a, da = expected(xd, gud[j * 2 * i:(j + 1) * 2 * i], [t], None, True)
        if quantize_acts:
            a, da = quantized(a, da)
        else:
            da = da + 2.0 ** -8 * (a.abs() + da)  # rounded to bf16
        wj = dnd[j * h:(j + 1) * h]
        z, dz = a @ wj.t(), da @ wj.abs().t() + sum_bound((a.abs() + da) @ wj.abs().t(), i)
        p = torch.from_numpy(np.where(ids == j, wts, 0.0).sum(1)).to(DEV).unsqueeze(1)
        want += p * z
        err += p * (dz + 2.0 ** -17 * (z.abs() + dz))  # the weight, and k products and sums
    check(y, want, err, torch.float32)


@pytest.mark.parametrize("shape, tile", mx_stream_shapes.STREAMED)
@pytest.mark.parametrize("swiglu", [False, True])
def test_w_past_the_caches(nv, shape, tile, swiglu):
    sizes, n, k = shape
    print(sizes[:4], n, k, tile, swiglu, flush=True)
    total = sum(sizes)
    a, ad, w, wd = operands(nv, n, total // 2 + 1, len(sizes) * n, k, "mx")
    rows = torch.randint(-1, total // 2 + 2, (total,), generator=gen(1), device=DEV).to(torch.int32)  # some outside A
    want, err = expected(ad, wd, sizes, rows, swiglu)
    for dt in (torch.float32, torch.bfloat16):
        check(nv.mx_grouped_gemm(a, w, offsets_of(sizes), rows=rows, swiglu=swiglu, dtype=dt), want, err, dt)
    if swiglu and want.shape[1] % 32 == 0:
        q = nv.mx_grouped_gemm(a, w, offsets_of(sizes), rows=rows, swiglu=True, out=nv.MXFP4Tensor.empty(total, want.shape[1], DEV))
        same = nv.mx_quantize(nv.mx_grouped_gemm(a, w, offsets_of(sizes), rows=rows, swiglu=True))
        assert torch.equal(q.codes, same.codes) and torch.equal(q.scales, same.scales)
