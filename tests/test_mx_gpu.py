"""The MXFP4 operators on the GPU against their plain float64 forms (tests/mx_ref.py)."""
import numpy as np
import pytest
import torch

import mx_ref
import synth
from gpu_util import DEV, padded, to_dev_bf16, to_dev_f16, to_dev_f32, to_dev_u8

pytestmark = pytest.mark.gpu
TDT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


def _np(t):
    return t.cpu().numpy()


def _bf16(v):
    """float array -> (device bf16 tensor, its values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16)
    return t.to(DEV), t.double().numpy()


def _weight(nv, rng, n, k, scale=0.02):
    codes, scales = mx_ref.quantize(rng.standard_normal((n, k)) * scale)
    return nv.MXFP4Tensor(to_dev_u8(codes), to_dev_u8(scales)), mx_ref.dequantize(codes, scales)


def _source(kind, v):
    """(device tensor, src_scale tensor or None, float64 values) of one source type."""
    if kind == "f32":
        return to_dev_f32(v), None, v.astype(np.float32).astype(np.float64)
    if kind == "bf16":
        t, d = _bf16(v)
        return t, None, d
    if kind == "f16":
        h = v.astype(np.float16)
        return to_dev_f16(h.view(np.uint16)), None, h.astype(np.float64)
    b, sc = synth.fp8_tensorwise(v.astype(np.float32))
    f = torch.from_numpy(b).view(torch.float8_e4m3fn).to(torch.float32).numpy()
    return to_dev_u8(b), torch.tensor([sc], dtype=torch.float32, device=DEV), (f * np.float32(sc)).astype(np.float64)


# ------------------------------------------------------------------------------------------------
# quantize, dequantize
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("pad", [0, 16])
@pytest.mark.parametrize("shape", [(1, 32), (1, 4096), (3, 96), (257, 160), (33, 2048), (1030, 544)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16", "e4m3"])
def test_quantize_matches_reference(nv, kind, shape, pad):
    rng = np.random.default_rng(shape[0] + pad)
    v = rng.standard_normal(shape) * np.exp2(rng.integers(-6, 6, (shape[0], 1)))
    if shape[0] > 2:
        v[1] = 0
    x, sc, d = _source(kind, v)
    q = nv.mx_quantize(padded(x, pad) if pad else x, src_scale=sc, check=True)
    codes, scales = mx_ref.quantize(d)
    assert np.array_equal(_np(q.scales), scales) and np.array_equal(_np(q.codes), codes)
    back = mx_ref.dequantize(codes, scales)
    assert np.array_equal(_np(nv.mx_dequantize(q, torch.float32)), back)
    out = torch.full((shape[0], shape[1] + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    nv.mx_dequantize(q, out=out[:, :shape[1]])
    assert np.array_equal(out[:, :shape[1]].double().cpu().numpy(), back)
    assert bool((out[:, shape[1]:] == 7).all())  # what lies between the rows stays


def test_quantize_every_exponent_ties_and_subnormals(nv):
    # one block per exponent: its grid points and midpoints and their neighbours, both signs
    base = np.array([4, 6, 7.96, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25], dtype=np.float32)
    pts = np.concatenate((base, np.nextafter(base, np.float32(0)), np.nextafter(base, np.float32(9))))
    pts = np.concatenate((pts, [-5, -0.25])).astype(np.float32)
    x = np.stack([np.ldexp(pts, e).astype(np.float32) for e in range(-147, 125)])
    x = np.concatenate((x, np.tile(np.array([[2.0 ** -149] + [0.0] * 31], np.float32), (1, 1)), -x[:4]))
    q = nv.mx_quantize(to_dev_f32(x), check=True)
    codes, scales = mx_ref.quantize(x.astype(np.float64))
    assert np.array_equal(_np(q.scales), scales)
    assert np.array_equal(_np(q.codes), codes)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_quantize_nonfinite_blocks(nv, kind):
    rng = np.random.default_rng(3)
    v = rng.standard_normal((6, 128))
    v[1, 40], v[2, 0], v[4, 127] = np.nan, np.inf, -np.inf
    x, _, d = _source(kind, v)
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = nv.mx_quantize(x, flags=flags)
    codes, scales = mx_ref.quantize(d)
    assert np.array_equal(_np(q.scales), scales) and np.array_equal(_np(q.codes), codes)
    assert int(flags.item()) == 1
    back = nv.mx_dequantize(q, torch.float32)
    assert np.array_equal(_np(back), mx_ref.dequantize(codes, scales), equal_nan=True)
    with pytest.raises(RuntimeError):
        nv.mx_quantize(x, check=True)


def test_dequantize_every_byte(nv):
    codes = np.tile(np.array([0x10, 0x32, 0x54, 0x76, 0x98, 0xBA, 0xDC, 0xFE] * 2, np.uint8), (1, 256))
    scales = np.arange(256, dtype=np.uint8)[None]
    q = nv.MXFP4Tensor(to_dev_u8(codes), to_dev_u8(scales))
    ref = mx_ref.dequantize(codes, scales)
    with np.errstate(over="ignore"):
        ref32 = ref.astype(np.float32)
    assert np.array_equal(_np(nv.mx_dequantize(q, torch.float32)), ref32, equal_nan=True)
    b = nv.mx_dequantize(q, torch.bfloat16).float().cpu().numpy()
    assert np.array_equal(b, torch.from_numpy(ref32).to(torch.bfloat16).float().numpy(), equal_nan=True)


def test_quantize_empty_and_long_strides(nv):
    assert nv.mx_quantize(torch.empty((0, 64), device=DEV)).shape == (0, 64)
    assert nv.mx_quantize(torch.empty((5, 0), device=DEV)).shape == (5, 0)
    buf = torch.randn((3, 1 << 20), device=DEV)
    q = nv.mx_quantize(buf[:, :64])
    codes, scales = mx_ref.quantize(buf[:, :64].double().cpu().numpy())
    assert np.array_equal(_np(q.codes), codes) and np.array_equal(_np(q.scales), scales)


# ------------------------------------------------------------------------------------------------
# product
# ------------------------------------------------------------------------------------------------
def _check_gemm(nv, a, w, wd, ad, out):
    m, n, k = ad.shape[0], wd.shape[0], wd.shape[1]
    c = nv.mx_gemm(a, w, dtype=TDT[out])
    ref = ad @ wd.T
    tol = mx_ref.fp32_sum_bound(np.abs(ad) @ np.abs(wd).T, k) + mx_ref.half_step(out, ref)
    err = np.abs(c.double().cpu().numpy() - ref)
    assert c.dtype == TDT[out] and tuple(c.shape) == (m, n)
    assert (err <= tol).all(), (m, n, k, float((err / tol).max()))
    return c


def _acts(nv, rng, m, k, act):
    v = rng.standard_normal((m, k))
    v[:, rng.integers(0, k)] *= 20
    a, d = _bf16(v)
    if act == "bf16":
        return a, d
    q = nv.mx_quantize(a)
    return q, mx_ref.dequantize(*mx_ref.quantize(d))


GEMM_SHAPES = [(1, 1, 32), (1, 4099, 4096), (2, 48, 96), (3, 17, 480), (5, 300, 512), (8, 64, 544), (13, 1000, 1056),
               (16, 16, 12288), (2, 5000, 608), (15, 8200, 544), (16, 17001, 160), (4, 12300, 6176),
               # up to 4, 8 and 16 rows; one, two and many groups of a wave, with and without a rest
               (1, 40, 7200), (4, 100, 2560), (6, 200, 4608), (7, 4200, 1536), (8, 12290, 4128), (9, 60, 2048),
               (11, 4200, 5152), (13, 96, 12288), (16, 8300, 4096), (16, 12300, 4128), (16, 12300, 2560),
               (17, 33, 160), (31, 129, 2048), (33, 200, 608), (48, 77, 1024), (64, 512, 96),
               (65, 1, 32), (65, 130, 96), (100, 257, 544), (128, 128, 1024), (129, 385, 480), (256, 512, 256),
               (257, 300, 768), (300, 515, 2080), (512, 96, 12288), (700, 1030, 160)]


@pytest.mark.parametrize("shape", GEMM_SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("act", ["mx", "bf16"])
def test_gemm(nv, act, shape):
    m, n, k = shape
    rng = np.random.default_rng(m * 7 + n)
    w, wd = _weight(nv, rng, n, k)
    a, ad = _acts(nv, rng, m, k, act)
    f = _check_gemm(nv, a, w, wd, ad, "f32")
    b = _check_gemm(nv, a, w, wd, ad, "bf16")
    assert torch.equal(f.to(torch.bfloat16), b)  # the same sums, rounded once
    assert torch.equal(f, nv.mx_gemm(a, w))      # and the same on every call


@pytest.mark.parametrize("m", [4, 40, 150])
@pytest.mark.parametrize("act", ["mx", "bf16"])
def test_gemm_one_hot_rows_reproduce_the_weight(nv, act, m):
    # row i selects column i: exact, so every element of W passes through at its place
    k, n = 192, 75
    rng = np.random.default_rng(m)
    w, wd = _weight(nv, rng, n, k)
    cols = rng.permutation(k)[:m] if m <= k else rng.integers(0, k, m)
    v = np.zeros((m, k))
    v[np.arange(m), cols] = 4.0
    a, _ = _bf16(v)
    c = nv.mx_gemm(nv.mx_quantize(a) if act == "mx" else a, w)
    assert np.array_equal(c.double().cpu().numpy(), 4.0 * wd[:, cols].T)


@pytest.mark.parametrize("m", [3, 130])
def test_gemm_strided_operands_leave_the_rest(nv, m):
    rng = np.random.default_rng(m)
    n, k = 77, 160
    w, wd = _weight(nv, rng, n, k)
    a, ad = _bf16(rng.standard_normal((m, k)))
    for dt, ldc in ((torch.float32, 81), (torch.bfloat16, 79)):
        buf = torch.full((m + 2, ldc), 3.0, dtype=dt, device=DEV)
        nv.mx_gemm(padded(a, 24), w, out=buf[1:m + 1, 1:n + 1])
        assert torch.equal(buf[1:m + 1, 1:n + 1], nv.mx_gemm(a, w, dtype=dt))
        rest = buf.clone()
        rest[1:m + 1, 1:n + 1] = 3
        assert bool((rest == 3).all())


@pytest.mark.parametrize("m", [5, 20, 70, 200])
@pytest.mark.parametrize("act", ["mx", "bf16"])
def test_gemm_nonfinite_stays_in_its_row_and_column(nv, act, m):
    rng = np.random.default_rng(m)
    n, k = 70, 320
    v = rng.standard_normal((m, k))
    clean, _ = _bf16(v)
    v[1, 100], v[3, 319] = np.nan, np.inf
    a, _ = _bf16(v)
    w, _ = _weight(nv, rng, n, k)
    if act == "mx":
        a, clean = nv.mx_quantize(a), nv.mx_quantize(clean)
    good = nv.mx_gemm(clean, w)
    w.scales[9, 4] = 255
    c = nv.mx_gemm(a, w)
    keep = torch.ones((m, n), dtype=torch.bool, device=DEV)
    keep[[1, 3]] = False
    keep[:, 9] = False
    assert bool((~torch.isfinite(c[1])).all()) and bool(torch.isnan(c[:, 9]).all())
    nz = nv.mx_dequantize(w, torch.float32)[:, 319] != 0  # inf times a zero code is NaN, which is not finite either
    assert bool((~torch.isfinite(c[3][nz])).all())
    assert torch.equal(c[keep], good[keep])


@pytest.mark.parametrize("m", [2, 66])
@pytest.mark.parametrize("act", ["mx", "bf16"])
def test_gemm_every_weight_scale(nv, act, m):
    # one column of C per scale byte: 4 x (1 + .5 + ...) summed exactly, scaled by 2^(b - 127)
    codes = np.tile(np.array([0x21, 0x43, 0x65, 0x07] * 4, np.uint8), (255, 1))
    scales = np.arange(255, dtype=np.uint8)[:, None]
    w = nv.MXFP4Tensor(to_dev_u8(codes), to_dev_u8(scales))
    a, _ = _bf16(np.full((m, 32), 0.25))
    c = nv.mx_gemm(nv.mx_quantize(a) if act == "mx" else a, w)
    with np.errstate(over="ignore"):
        ref = (0.25 * mx_ref.dequantize(codes, scales).sum(axis=1)).astype(np.float32)
    got = _np(c)
    normal = np.abs(ref) >= 2.0 ** -120  # products below the normal range may be flushed
    ok = normal & (scales[:, 0] <= 250)  # a bf16 operand of 6 x 2^127 overflows in the expanded form
    assert np.array_equal(got[:, ok], np.tile(ref[ok], (m, 1)))
    assert np.abs(got[:, ~normal]).max() <= 2.0 ** -120


def test_gemm_empty(nv):
    w, _ = _weight(nv, np.random.default_rng(0), 8, 64)
    assert nv.mx_gemm(torch.empty((0, 64), dtype=torch.bfloat16, device=DEV), w).shape == (0, 8)
    none = nv.MXFP4Tensor.empty(0, 64, DEV)
    assert nv.mx_gemm(torch.zeros((3, 64), dtype=torch.bfloat16, device=DEV), none).shape == (3, 0)
    k0 = nv.MXFP4Tensor.empty(8, 0, DEV)
    out = torch.full((70, 8), 5.0, device=DEV)
    nv.mx_gemm(torch.empty((70, 0), dtype=torch.bfloat16, device=DEV), k0, out=out)
    assert bool((out == 0).all())


def test_gemm_less_workspace_runs_unsplit(nv):
    from bit_gemm_nvfp4_amd import mx
    rng = np.random.default_rng(5)
    m, n, k = 128, 256, 12288
    w, wd = _weight(nv, rng, n, k)
    a, ad = _acts(nv, rng, m, k, "mx")
    assert nv.mx_workspace_size(mx.MX_OP_GEMM_MX, m, n, k) > 0  # the planned form splits K
    c = nv.mx_gemm(a, w, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    tol = mx_ref.fp32_sum_bound(np.abs(ad) @ np.abs(wd).T, k) + mx_ref.half_step("f32", ad @ wd.T)
    assert (np.abs(c.double().cpu().numpy() - ad @ wd.T) <= tol).all()


# ------------------------------------------------------------------------------------------------
# experts
# ------------------------------------------------------------------------------------------------
def _moe_case(nv, seed, t, e, h, i, logits=None, ldt=torch.float32):
    rng = np.random.default_rng(seed)
    gu, gud = _weight(nv, rng, e * 2 * i, h, 0.05)
    dn, dnd = _weight(nv, rng, e * h, i, 0.05)
    x, xd = _bf16(rng.standard_normal((t, h)))
    lg = rng.standard_normal((t, e)) * 2 if logits is None else logits
    lt = torch.from_numpy(np.asarray(lg, dtype=np.float32)).to(ldt)
    return x, xd, lt.to(DEV), lt.double().numpy(), gu, gud, dn, dnd


def _check_moe(nv, case, e, k, renorm, out="bf16"):
    x, xd, lt, ld, gu, gud, dn, dnd = case
    y, ids, wts = nv.mx_moe(x, lt, gu, dn, k, renormalize=renorm, dtype=TDT[out], routing=True)
    ref, bound, rids, rw = mx_ref.moe(xd, ld, gud, dnd, e, k, renorm)
    assert np.array_equal(_np(ids), rids)
    good = np.isfinite(ref).all(axis=1)
    # exp of a difference rounded to fp32: relative 2^-24 times the difference (at most 2^6 here), and the sum
    assert (np.abs(_np(wts).astype(np.float64) - rw) <= 2.0 ** -17 * np.abs(rw))[good].all()
    got = y.double().cpu().numpy()
    assert np.isnan(got[~good]).all()
    tol = bound + 2.0 ** -17 * np.abs(ref) + mx_ref.half_step(out, ref)
    err = np.abs(got - ref)[good]
    assert (err <= tol[good]).all(), float((err / tol[good]).max())
    return y


MOE_CASES = [(1, 8, 2, 64, 32), (1, 1, 1, 32, 32), (1, 64, 8, 512, 96), (2, 5, 5, 96, 160), (3, 16, 3, 544, 64),
             (7, 4, 2, 128, 544), (16, 8, 2, 256, 64), (17, 130, 4, 64, 32), (33, 12, 3, 160, 96), (64, 8, 4, 96, 64),
             (64, 512, 16, 32, 32), (50, 3, 1, 1056, 32),
             (64, 2, 2, 160, 1056), (12, 3, 2, 96, 544), (5, 4, 2, 1536, 416), (3, 6, 2, 2048, 288),
             (9, 4, 2, 832, 160), (40, 8, 4, 4128, 96), (2, 1, 1, 32, 512)]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("case", MOE_CASES, ids=lambda s: "x".join(map(str, s)))
def test_moe(nv, case, renorm):
    t, e, k, h, i = case
    c = _moe_case(nv, t * 100 + e, t, e, h, i)
    y = _check_moe(nv, c, e, k, renorm)
    _check_moe(nv, c, e, k, renorm, "f32")
    assert torch.equal(y, nv.mx_moe(c[0], c[2], c[4], c[6], k, renormalize=renorm))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("t", [2, 9, 40])
def test_moe_masks_ties_and_nonfinite_logits(nv, t, renorm):
    e, k, h, i = 6, 3, 64, 64
    rng = np.random.default_rng(t)
    lg = np.round(rng.standard_normal((t, e)))  # many ties
    lg[rng.random((t, e)) < 0.3] = -np.inf
    lg[0] = -np.inf
    lg[0, 4] = -1e30  # one expert left
    lg[1] = -np.inf   # none
    if t > 4:
        lg[3, 2], lg[4, 0] = np.nan, np.inf
        lg[5] = np.finfo(np.float32).min  # the type's lowest value is a value, not a mask
        lg[6] = 1e30
    for ldt in (torch.float32, torch.bfloat16):
        _check_moe(nv, _moe_case(nv, t, t, e, h, i, lg, ldt), e, k, renorm)


def test_moe_all_tokens_choose_the_same_experts(nv):
    lg = np.tile(np.array([0.0, 3.0, 1.0, 2.0, -1.0]), (64, 1))
    _check_moe(nv, _moe_case(nv, 1, 64, 5, 128, 96, lg), 5, 2, True)


def test_moe_nonfinite_token_stays_in_its_row(nv):
    x, xd, lt, ld, gu, gud, dn, dnd = _moe_case(nv, 8, 20, 4, 96, 64)
    good = nv.mx_moe(x, lt, gu, dn, 2)
    x2 = x.clone()
    x2[7, 50] = float("nan")
    y = nv.mx_moe(x2, lt, gu, dn, 2)
    rows = [r for r in range(20) if r != 7]
    assert bool(torch.isnan(y[7]).all()) and torch.equal(y[rows], good[rows])


def test_moe_strided_views_and_empty(nv):
    x, _, lt, _, gu, _, dn, _ = _moe_case(nv, 2, 5, 4, 64, 32)
    ref = nv.mx_moe(x, lt, gu, dn, 2)
    buf = torch.full((6, 71), 9.0, dtype=torch.bfloat16, device=DEV)
    nv.mx_moe(padded(x, 8), padded(lt, 3), gu, dn, 2, out=buf[:5, 1:65])
    assert torch.equal(buf[:5, 1:65], ref)
    buf[:5, 1:65] = 9
    assert bool((buf == 9).all())
    assert nv.mx_moe(x[:0], lt[:0], gu, dn, 2).shape == (0, 64)


# ------------------------------------------------------------------------------------------------
# together, streams, graphs
# ------------------------------------------------------------------------------------------------
def _chain(nv, x, lt, wq, gu, dn):
    """A block as it is served: quantize, project, expert layer, project back."""
    h = nv.mx_gemm(nv.mx_quantize(x), wq, dtype=torch.bfloat16)
    y = nv.mx_moe(h, lt, gu, dn, 2)
    return nv.mx_gemm(y, wq), y


@pytest.mark.parametrize("t", [1, 24, 64])
def test_chain_against_reference(nv, t):
    rng = np.random.default_rng(t)
    e, h, i = 6, 128, 96
    x, xd, lt, ld, gu, gud, dn, dnd = _moe_case(nv, t, t, e, h, i)
    wq, wqd = _weight(nv, rng, h, h, 0.1)
    out, y = _chain(nv, x, lt, wq, gu, dn)
    hd = nv.mx_gemm(nv.mx_quantize(x), wq, dtype=torch.bfloat16)
    href = mx_ref.dequantize(*mx_ref.quantize(xd)) @ wqd.T
    assert (np.abs(hd.double().cpu().numpy() - href) <= 2.0 ** -8 * np.abs(href) + 1e-5).all()
    yref, bound, _, _ = mx_ref.moe(hd.double().cpu().numpy(), ld, gud, dnd, e, 2, True)
    yd = y.double().cpu().numpy()
    assert (np.abs(yd - yref) <= bound + (2.0 ** -17 + 2.0 ** -8) * np.abs(yref) + 1e-30).all()
    ref = yd @ wqd.T
    tol = mx_ref.fp32_sum_bound(np.abs(yd) @ np.abs(wqd).T, h) + mx_ref.half_step("f32", ref)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()


def test_side_stream_and_threads_of_work(nv):
    x, _, lt, _, gu, _, dn, _ = _moe_case(nv, 4, 12, 6, 128, 96)
    wq, _ = _weight(nv, np.random.default_rng(9), 128, 128, 0.1)
    big, _ = _bf16(np.random.default_rng(2).standard_normal((300, 128)))
    ref, refb = _chain(nv, x, lt, wq, gu, dn)[0], nv.mx_gemm(big, wq)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:  # two streams at a time, each call with its own workspace
        with torch.cuda.stream(s):
            outs.append((_chain(nv, x, lt, wq, gu, dn)[0], nv.mx_gemm(big, wq)))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, ref) and torch.equal(b, refb)


def test_graph_replays_with_kept_workspaces(nv):
    from bit_gemm_nvfp4_amd import mx
    t, e, h, i = 10, 6, 128, 96
    x, _, lt, _, gu, _, dn, _ = _moe_case(nv, 4, t, e, h, i)
    wl, _ = _weight(nv, np.random.default_rng(9), 200, 12288, 0.1)
    big, _ = _bf16(np.random.default_rng(2).standard_normal((130, 12288)))
    ws_moe = nv.mx_moe_workspace(t, 2, gu, dn)
    ws_g = nv.mx_gemm_workspace(big, wl)
    qb = nv.mx_quantize(big)
    ws_q = nv.mx_gemm_workspace(qb, wl)
    s = torch.cuda.Stream()
    outs = {}

    def work():
        q = nv.mx_quantize(big, out=qb)
        outs["y"] = nv.mx_moe(x, lt, gu, dn, 2, workspace=ws_moe)
        outs["c"] = nv.mx_gemm(big, wl, workspace=ws_g)
        outs["cq"] = nv.mx_gemm(q, wl, workspace=ws_q)
        outs["d"] = nv.mx_dequantize(q)
    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs that share the workspaces
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            work()
        graphs.append((g, dict(outs)))
    rng = np.random.default_rng(11)
    for rep in range(4):
        x.copy_(_bf16(rng.standard_normal((t, h)))[0])
        lt.copy_(torch.from_numpy(rng.standard_normal((t, e)).astype(np.float32)))
        big.copy_(_bf16(rng.standard_normal((130, 12288)))[0])
        torch.cuda.synchronize()
        g, o = graphs[rep % 2]
        g.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in o.items()}
        q = nv.mx_quantize(big)
        assert torch.equal(got["y"], nv.mx_moe(x, lt, gu, dn, 2))
        assert torch.equal(got["c"], nv.mx_gemm(big, wl))
        assert torch.equal(got["cq"], nv.mx_gemm(q, wl))
        assert torch.equal(got["d"], nv.mx_dequantize(q))


def test_int64_offsets(nv):
    # a weight whose codes pass 2^31 bytes, and an activation buffer whose rows lie far apart
    rows, k = (1 << 20) + 40, 4096
    codes = torch.zeros((rows, k // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((rows, k // 32), 127, dtype=torch.uint8, device=DEV)
    codes[rows - 1] = 0x22
    codes[7] = 0x44
    w = nv.MXFP4Tensor(codes, scales)
    for m in (1, 16, 17, 66):
        a = torch.ones((m, k), dtype=torch.bfloat16, device=DEV)
        c = nv.mx_gemm(a, w, dtype=torch.bfloat16)
        assert bool((c[:, rows - 1] == k).all()) and bool((c[:, 7] == 2 * k).all())
        assert int((c != 0).sum()) == 2 * m
    d = nv.mx_dequantize(w)
    assert bool((d[rows - 1] == 1).all()) and bool((d[7] == 2).all())
    del d
    far = torch.zeros((3, (1 << 30) + 64), dtype=torch.bfloat16, device=DEV)
    far[:, :k] = 1
    assert bool((nv.mx_gemm(far[:, :k], w, dtype=torch.bfloat16)[:, rows - 1] == k).all())
    assert bool((nv.mx_dequantize(nv.mx_quantize(far[:, :k])) == 1).all())


# one token over many experts, and two tokens per expert (the tall down product), H beyond the register form
@pytest.mark.parametrize("case", [(1, 96, 4096, 12288), (64, 32, 8192, 16896)], ids=lambda s: "x".join(map(str, s)))
def test_moe_int64_offsets(nv, case):
    t, e, h, i = case

    def zeros(rows, cols):
        return nv.MXFP4Tensor(torch.zeros((rows, cols // 2), dtype=torch.uint8, device=DEV),
                              torch.full((rows, cols // 32), 127, dtype=torch.uint8, device=DEV))
    gu, dn = zeros(e * 2 * i, h), zeros(e * h, i)
    assert gu.codes.numel() > 2 ** 31 and dn.codes.numel() > 2 ** 31
    # the last expert: inner element i - 1 is silu(1) * 1, output element h - 1 takes it
    gu.codes[(e - 1) * 2 * i + i - 1, 0] = 0x02
    gu.codes[e * 2 * i - 1, 0] = 0x02
    dn.codes[e * h - 1, i // 2 - 1] = 0x20
    x = torch.zeros((t, h), dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    logits = torch.zeros((t, e), device=DEV)
    logits[:, e - 1] = 1
    y = nv.mx_moe(x, logits, gu, dn, 1, dtype=torch.float32).double().cpu().numpy()
    want = 1 / (1 + np.exp(-1.0))
    # two planes of h (2^-17) and a few fp32 roundings (exp, quotient, product, sums with zeros)
    assert (np.abs(y[:, h - 1] - want) <= want * (2.0 ** -17 + 8 * 2.0 ** -24)).all()
    assert (y[:, :h - 1] == 0).all()
