"""Router, products grouped by rows, weighted sum and the expert layer for any number of tokens, on the GPU against
their plain float64 forms."""
import numpy as np
import pytest
import torch

import mx_group_shapes
import mx_ref
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


def half_step(t, ref):
    """Largest rounding of float64 `ref` to the output type, and of what lies below its smallest normal number."""
    return ref.abs() * torch.finfo(t).eps / 2 + torch.finfo(t).tiny


def sum_bound(absprod, k):
    """Bound on an fp32 sum of k products whose magnitudes add up to absprod: a partial sum is at most absprod and is
    rounded at most once per eight products, and 16 more times in the joins."""
    return (k / 8 + 16) * 2.0 ** -24 * absprod


# ------------------------------------------------------------------------------------------------
# router and sort
# ------------------------------------------------------------------------------------------------
def sort_reference(ids, groups):
    """(offsets, rows, places) of ids [T, k], by a stable sort on the host."""
    t, k = ids.shape
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < groups)
    order = np.argsort(np.where(ok, flat, groups), kind="stable")
    n = int(ok.sum())
    rows, places = np.full(t * k, -1), np.full(t * k, -1)
    rows[:n] = order[:n] // k
    places[order[:n]] = np.arange(n)
    offsets = np.searchsorted(np.sort(flat[ok], kind="stable"), np.arange(groups + 1))
    return offsets, rows, places.reshape(t, k)


def check_sort(r, ids, groups):
    offsets, rows, places = sort_reference(ids, groups)
    assert np.array_equal(r.offsets.cpu().numpy(), offsets)
    assert np.array_equal(r.rows.cpu().numpy(), rows)
    assert np.array_equal(r.places.cpu().numpy(), places)


# one workgroup up to 16 rows, then 16 rows a workgroup, more from 4096 rows on; 64, 128, 256 and 512 experts to a row
@pytest.mark.parametrize("t, e, k", [(1, 1, 1), (1, 64, 8), (3, 65, 2), (16, 40, 3), (17, 5, 5), (64, 128, 16), (65, 130, 3), (300, 512, 16),
                                     (1000, 257, 6), (4096, 40, 1), (4097, 7, 2), (9000, 33, 4)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(nv, t, e, k, dt, renorm):
    g = gen(t + e)
    logits = (randn(g, t, e) * 2).to(TDT[dt])
    logits[torch.rand((t, e), generator=g, device=DEV) < 0.2] = float("-inf")
    if t > 2:
        logits[t // 2] = float("-inf")
        logits[t // 3] = 0.25  # ties everywhere
        logits[t - 1, 0] = float("nan")
        logits[0, e - 1] = float("inf")
    if t > 16:
        logits[5, :] = -3e38
        logits[6, 0], logits[6, 1:] = 0.0, -0.0
        logits[7, e // 2] = -float("nan")
    r = nv.mx_route(padded(logits, 3) if t % 2 else logits, k, renormalize=renorm)
    lg = logits.double().cpu().numpy()
    ids, wts = mx_ref.route(lg, k, renorm)
    bad = np.isnan(lg).any(axis=1) | (lg == np.inf).any(axis=1)
    wts[bad] = np.nan
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    # exp of a rounded difference (|d| 2^-24 and a step or two), a sum of e terms in a tree, a division: all relative
    fin = np.where(np.isfinite(lg), lg, 0)
    tol = (2 * (fin.max(axis=1) - fin.min(axis=1)).clip(max=104) + 40) * 2.0 ** -24
    got = r.weights.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(wts))
    err = np.abs(np.nan_to_num(got) - np.nan_to_num(wts))
    assert (err <= tol[:, None] * np.nan_to_num(wts) + 2.0 ** -126).all()
    check_sort(r, ids, e)


@pytest.mark.parametrize("t, k, groups", [(1, 1, 1), (5, 3, 4), (64, 1, 512), (100, 7, 3), (4096, 1, 64), (4097, 1, 64), (20000, 3, 300),
                                          (1 << 20, 2, 40)])
def test_group_rows(nv, t, k, groups):
    rng = np.random.default_rng(t)
    ids = rng.integers(-1, groups + 1, (t, k)).astype(np.int32)  # no choice on either side, a group twice in a row
    if t > 4:
        ids[1], ids[2], ids[3, 0] = 2 ** 31 - 1, -2 ** 31, groups - 1
        ids[t // 2:t // 2 + t // 4] = 0  # a long run of one group
    check_sort(nv.mx_group_rows(torch.from_numpy(ids).to(DEV), groups), ids, groups)


def test_group_rows_without_rows_or_choices(nv):
    r = nv.mx_group_rows(torch.empty((0, 2), dtype=torch.int32, device=DEV), 5)
    assert r.offsets.tolist() == [0] * 6 and r.rows.numel() == 0
    r = nv.mx_group_rows(torch.full((9,), -1, dtype=torch.int32, device=DEV), 5)
    assert r.offsets.tolist() == [0] * 6 and r.rows.tolist() == [-1] * 9 and r.places.flatten().tolist() == [-1] * 9
    r = nv.mx_route(torch.empty((0, 4), device=DEV), 2)
    assert r.offsets.tolist() == [0] * 5 and r.ids.shape == (0, 2)


# ------------------------------------------------------------------------------------------------
# grouped products
# ------------------------------------------------------------------------------------------------
def operands(nv, seed, a_rows, w_rows, k, act):
    """(a, its float64 values, w, its float64 values)."""
    g = gen(seed)
    x = randn(g, a_rows, k).to(torch.bfloat16)
    w = nv.mx_quantize(randn(g, w_rows, k) * 0.05)
    wd = nv.mx_dequantize(w, torch.float32).double()
    if act == "mx":
        a = nv.mx_quantize(x)
        return a, nv.mx_dequantize(a, torch.float32).double(), w, wd
    return x, x.double(), w, wd


def expected(ad, wd, sizes, rows, swiglu):
    """(float64 C of the grouped rows, bound on the error before its rounding)."""
    n = wd.shape[0] // len(sizes)
    k = wd.shape[1]
    outs, errs, lo = [], [], 0
    for j, size in enumerate(sizes):
        part = ad[lo:lo + size] if rows is None else torch.where(
            ((rows[lo:lo + size] >= 0) & (rows[lo:lo + size] < ad.shape[0])).unsqueeze(1),
            ad[rows[lo:lo + size].long().clamp(0, ad.shape[0] - 1)], 0.0)
        wj = wd[j * n:(j + 1) * n]
        v, mag = part @ wj.t(), part.abs() @ wj.abs().t()
        dv = sum_bound(mag, k)
        if swiglu:
            gate, up, dg, du = v[:, :n // 2], v[:, n // 2:], dv[:, :n // 2], dv[:, n // 2:]
            s = gate / (1 + torch.exp(-gate))
            v = s * up
            # |silu'| < 1.1; exp, a sum, a division and a product of fp32 values: a few steps
            dv = 1.1 * dg * (up.abs() + du) + s.abs() * du + 2.0 ** -20 * v.abs()
        outs.append(v)
        errs.append(dv)
        lo += size
    return torch.cat(outs), torch.cat(errs)


def check(got, want, err, dt):
    diff = (got.double() - want).abs()
    assert bool((diff <= err + half_step(dt, want) + err * torch.finfo(dt).eps).all()), float((diff - err).max())


def offsets_of(sizes):
    return torch.tensor(np.concatenate(([0], np.cumsum(sizes))), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["bf16", "mx"])
@pytest.mark.parametrize("sizes, n, k", [([1], 2, 32), ([0, 5], 34, 64), ([17, 0, 0, 3, 40], 130, 544), ([1] * 70 + [0] * 3 + [9], 64, 96),
                                         ([300, 0, 45], 258, 1056), ([3, 130, 1], 1002, 4096)])
def test_grouped_products(nv, sizes, n, k, act, out, gather, swiglu):
    print(sizes[:6], n, k, act, out, gather, swiglu, flush=True)
    rows_n = sum(sizes)
    a_rows = 37 if gather else rows_n
    a, ad, w, wd = operands(nv, n + k, a_rows, len(sizes) * n, k, act)
    rows = None
    if gather:
        rows = torch.randint(-2, a_rows + 2, (rows_n,), generator=gen(k), device=DEV).to(torch.int32)  # some outside A
    got = nv.mx_grouped_gemm(a, w, offsets_of(sizes), rows=rows, swiglu=swiglu, dtype=TDT[out])
    want, err = expected(ad, wd, sizes, rows, swiglu)
    assert got.dtype is TDT[out] and got.shape == want.shape
    check(got, want, err, TDT[out])


@pytest.mark.parametrize("shape, act, tile", mx_group_shapes.GROUPED)
@pytest.mark.parametrize("swiglu", [False, True])
def test_every_tile_shape(nv, shape, act, tile, swiglu):
    sizes, n, k = shape
    print(shape, act, tile, flush=True)
    total = sum(sizes)
    a_rows = total // 2 + 1
    a, ad, w, wd = operands(nv, n, a_rows, len(sizes) * n, k, act)
    rows = torch.randint(0, a_rows, (total,), generator=gen(1), device=DEV).to(torch.int32)
    want, err = expected(ad, wd, sizes, rows, swiglu)
    for dt in TDT.values():
        check(nv.mx_grouped_gemm(a, w, offsets_of(sizes), rows=rows, swiglu=swiglu, dtype=dt), want, err, dt)
    if swiglu and want.shape[1] % 32 == 0:
        q = nv.MXFP4Tensor.empty(total, want.shape[1], DEV)
        nv.mx_grouped_gemm(a, w, offsets_of(sizes), rows=rows, swiglu=True, out=q)
        same = nv.mx_quantize(nv.mx_grouped_gemm(a, w, offsets_of(sizes), rows=rows, swiglu=True))
        assert torch.equal(q.codes, same.codes) and torch.equal(q.scales, same.scales)


@pytest.mark.parametrize("act", ["bf16", "mx"])
def test_grouped_mxfp4_output_is_the_quantized_fp32_one(nv, act):
    sizes, n, k = [70, 0, 1, 33], 192, 160
    a, _, w, _ = operands(nv, 4, sum(sizes), len(sizes) * n, k, act)
    if act == "bf16":
        a[3] = 0          # a block of zeros
        a[5, 7] = float("nan")
        a[6, 0] = 3e38    # infinities in its row
    offs = offsets_of(sizes)
    want = nv.mx_quantize(nv.mx_grouped_gemm(a, w, offs, swiglu=True))
    q = nv.MXFP4Tensor.empty(sum(sizes), n // 2, DEV)
    assert nv.mx_grouped_gemm(a, w, offs, swiglu=True, out=q) is q
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)


@pytest.mark.parametrize("act", ["bf16", "mx"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_rows_outside_the_groups_and_between_the_rows_stay(nv, act, swiglu):
    sizes, n, k = [4, 0, 66], 70, 96
    first, last = 3, 20  # rows before the first group and behind the last one
    total = first + sum(sizes) + last
    a, ad, w, wd = operands(nv, 9, total, len(sizes) * n, k, act)
    if act == "bf16":
        a = padded(a, 8)
    cols = n // 2 if swiglu else n
    buf = torch.full((total, cols + 5), 7.0, device=DEV)
    nv.mx_grouped_gemm(a, w, offsets_of(sizes) + first, swiglu=swiglu, out=buf[:, :cols])
    lo, hi = first, first + sum(sizes)
    want, err = expected(ad[lo:hi], wd, sizes, None, swiglu)
    check(buf[lo:hi, :cols], want, err, torch.float32)
    assert bool((buf[:lo] == 7).all()) and bool((buf[hi:] == 7).all()) and bool((buf[:, cols:] == 7).all())


def test_one_row_with_nan_or_infinity_stays_alone(nv):
    sizes, n, k = [40, 30], 64, 128
    a, ad, w, wd = operands(nv, 2, 70, 2 * n, k, "bf16")
    clean = nv.mx_grouped_gemm(a, w, offsets_of(sizes))
    a[11, 3], a[50, 0] = float("nan"), float("inf")
    got = nv.mx_grouped_gemm(a, w, offsets_of(sizes))
    keep = [i for i in range(70) if i not in (11, 50)]
    assert torch.equal(got[keep], clean[keep]) and bool((~got[[11, 50]].isfinite()).all())
    # a weight block that is NaN: its column in its own group
    w.scales[5, 1] = 255
    got = nv.mx_grouped_gemm(nv.mx_quantize(ad.to(torch.bfloat16)), w, offsets_of(sizes))
    nan = got.isnan()
    assert bool(nan[:40, 5].all()) and int(nan.sum()) == 40


def test_offsets_out_of_order_or_range_stay_within_c(nv):
    # values past the rows are cut off there, a group that ends before it starts has no rows
    n, k, total = 64, 64, 50
    a, ad, w, wd = operands(nv, 3, total, 3 * n, k, "mx")
    out = torch.full((total + 8, n), 5.0, device=DEV)
    nv.mx_grouped_gemm(a, w, torch.tensor([-7, 20, 10, 1 << 30], dtype=torch.int32, device=DEV), out=out[:total])
    want, err = expected(ad[:20], wd[:n], [20], None, False)
    check(out[:10], want[:10], err[:10], torch.float32)
    want, err = expected(ad[10:total], wd[2 * n:], [total - 10], None, False)
    check(out[20:total], want[10:], err[10:], torch.float32)
    assert bool((out[total:] == 5).all())


# ------------------------------------------------------------------------------------------------
# weighted sum, layer
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("zt", ["f32", "bf16"])
@pytest.mark.parametrize("yt", ["f32", "bf16"])
@pytest.mark.parametrize("t, k, p, cols", [(1, 1, 1, 1), (3, 2, 9, 37), (70, 8, 200, 256), (5, 16, 30, 4100)])
def test_combine(nv, t, k, p, cols, zt, yt):
    g = gen(t * k)
    z = randn(g, p, cols).to(TDT[zt])
    places = torch.randint(-2, p + 2, (t, k), generator=g, device=DEV).to(torch.int32)
    weights = torch.rand((t, k), generator=g, device=DEV)
    ok = (places >= 0) & (places < p)
    zd = torch.where(ok.unsqueeze(2), z.double()[places.long().clamp(0, p - 1)], 0.0)
    terms = zd * weights.double().unsqueeze(2)
    want, err = terms.sum(1), 2 * k * 2.0 ** -24 * terms.abs().sum(1)
    buf = torch.full((t, cols + 3), 7.0, dtype=TDT[yt], device=DEV)
    check(nv.mx_combine(z, places, weights, dtype=TDT[yt]), want, err, TDT[yt])
    nv.mx_combine(padded(z, 8 - cols % 8), places, weights, out=buf[:, :cols])
    check(buf[:, :cols], want, err, TDT[yt])
    assert bool((buf[:, cols:] == 7).all())


def test_combine_leaves_out_rows_without_a_place(nv):
    z = torch.full((2, 40), float("nan"), device=DEV)
    z[1] = 3
    places = torch.tensor([[1, -1], [-1, -1], [-1, 1]], dtype=torch.int32, device=DEV)
    weights = torch.tensor([[0.5, 0.0], [0.0, 0.0], [float("nan"), 1.0]], device=DEV)
    y = nv.mx_combine(z, places, weights, dtype=torch.float32)
    assert bool((y[0] == 1.5).all()) and bool((y[1] == 0).all()) and bool(y[2].isnan().all())


def experts(nv, seed, t, e, h, i, scale=0.1):
    g = gen(seed)
    x = randn(g, t, h).to(torch.bfloat16)
    logits = randn(g, t, e) * 2
    if t > 4:
        logits[t // 2] = float("-inf")
        logits[1, torch.arange(e, device=DEV) % 3 > 0] = float("-inf")
    return x, logits, nv.mx_quantize(randn(g, e * 2 * i, h) * scale), nv.mx_quantize(randn(g, e * h, i) * scale)


@pytest.mark.parametrize("quantize_acts", [False, True])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("t, e, k, h, i", [(1, 4, 2, 64, 32), (65, 8, 3, 96, 64), (300, 70, 4, 160, 96), (700, 3, 1, 256, 128)])
def test_layer_is_its_calls_one_after_the_other(nv, t, e, k, h, i, dt, quantize_acts):
    x, logits, gu, dn = experts(nv, t, t, e, h, i)
    y, ids, wts = nv.mx_experts(x, logits, gu, dn, k, quantize_acts=quantize_acts, dtype=TDT[dt], routing=True)
    r = nv.mx_route(logits, k)
    assert torch.equal(ids, r.ids) and torch.equal(wts, r.weights)
    if quantize_acts:
        hid = nv.MXFP4Tensor.empty(t * k, i, DEV)
        hid.codes.zero_()
        hid.scales.zero_()
        nv.mx_grouped_gemm(nv.mx_quantize(x), gu, r.offsets, rows=r.rows, swiglu=True, out=hid)
    else:
        hid = nv.mx_grouped_gemm(x, gu, r.offsets, rows=r.rows, swiglu=True, out=torch.zeros((t * k, i), dtype=torch.bfloat16, device=DEV))
    z = nv.mx_grouped_gemm(hid, dn, r.offsets, out=torch.zeros((t * k, h), dtype=TDT[dt], device=DEV))
    assert torch.equal(y, nv.mx_combine(z, r.places, r.weights, dtype=TDT[dt]))
    if t > 4:
        assert bool((y[t // 2] == 0).all())


@pytest.mark.parametrize("renorm", [True, False])
def test_layer_against_float64(nv, renorm):
    t, e, k, h, i = 130, 6, 2, 128, 96
    x, logits, gu, dn = experts(nv, 8, t, e, h, i)
    logits[9, 2] = float("nan")
    y = nv.mx_experts(x, logits, gu, dn, k, renormalize=renorm, quantize_acts=False, dtype=torch.float32)
    gud, dnd = nv.mx_dequantize(gu, torch.float32).double(), nv.mx_dequantize(dn, torch.float32).double()
    ids, wts = mx_ref.route(logits.double().cpu().numpy(), k, renorm)
    want, err, xd = torch.zeros((t, h), dtype=torch.float64, device=DEV), torch.zeros((t, h), dtype=torch.float64, device=DEV), x.double()
    for j in range(e):
        a, da = expected(xd, gud[j * 2 * i:(j + 1) * 2 * i], [t], None, True)
        da = da + 2.0 ** -8 * a.abs()  # h is rounded to bf16
        wj = dnd[j * h:(j + 1) * h]
        z, dz = a @ wj.t(), da @ wj.abs().t() + sum_bound((a.abs() + da) @ wj.abs().t(), i)
        p = torch.from_numpy(np.where(ids == j, wts, 0.0).sum(1)).to(DEV).unsqueeze(1)
        want += p * z
        err += p * (dz + 2.0 ** -18 * z.abs())
    keep = [r for r in range(t) if r != 9]
    check(y[keep], want[keep], err[keep], torch.float32)
    assert bool(y[9].isnan().all())


def test_layer_agrees_with_the_one_for_few_tokens(nv):
    t, e, k, h, i = 40, 8, 2, 256, 128
    x, logits, gu, dn = experts(nv, 3, t, e, h, i)
    few = nv.mx_moe(x, logits, gu, dn, k, dtype=torch.float32)
    any_ = nv.mx_experts(x, logits, gu, dn, k, quantize_acts=False, dtype=torch.float32)
    # they differ by the rounding of h to bf16: 2^-8 of each of its values at most
    gud, dnd = nv.mx_dequantize(gu, torch.float32), nv.mx_dequantize(dn, torch.float32)
    ids, wts = mx_ref.route(logits.double().cpu().numpy(), k, True)
    bound = torch.zeros((t, h), device=DEV)
    for j in range(e):
        v = x.float() @ gud[j * 2 * i:(j + 1) * 2 * i].t()
        a = (v[:, :i] * torch.sigmoid(v[:, :i]) * v[:, i:]).abs() @ dnd[j * h:(j + 1) * h].abs().t()
        bound += torch.from_numpy(np.where(ids == j, wts, 0.0).sum(1)).float().to(DEV).unsqueeze(1) * a
    assert bool(((few - any_).abs() <= 1.01 * 2.0 ** -8 * bound + 2.0 ** -14 * bound).all())


def test_many_rows_and_experts(nv):
    """A router's plan used as it comes: 20000 tokens over 128 experts, against float64 on a sample of the rows."""
    t, e, k, h, i = 20000, 128, 2, 128, 64
    x, logits, gu, dn = experts(nv, 5, t, e, h, i)
    r = nv.mx_route(logits, k)
    got = nv.mx_grouped_gemm(x, gu, r.offsets, rows=r.rows, swiglu=True, dtype=torch.float32)
    gud = nv.mx_dequantize(gu, torch.float32).double()
    offs = r.offsets.tolist()
    for j in (0, 1, 63, 64, 100, 127):
        lo, hi = offs[j], offs[j + 1]
        want, err = expected(x.double(), gud[j * 2 * i:(j + 1) * 2 * i], [hi - lo], r.rows[lo:hi], True)
        check(got[lo:hi], want, err, torch.float32)
