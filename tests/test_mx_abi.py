"""The MXFP4 entry points on the CPU: header and exports, refusals before anything touches the GPU, and
pins of the plain float64 forms the GPU tests compare against."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import mx_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


def _mx(nv, rows, cols, codes=FAKE, scales=FAKE):
    from bit_gemm_nvfp4_amd.mx import CMXTensor
    return CMXTensor(codes, scales, rows, cols)


def test_header_exports_and_binding_agree(nv):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "mxfp4.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(nv.MX_EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", nv.LIB_PATH], capture_output=True, text=True).stdout
    assert set(declared) <= set(re.findall(r"\bT (\w+)$", out, flags=re.M))


def test_workspace_sizes(nv):
    from bit_gemm_nvfp4_amd import mx
    assert nv.mx_workspace_size(mx.MX_OP_GEMM_MX, 16, 4096, 12288) == 0
    assert nv.mx_workspace_size(mx.MX_OP_GEMM_BF16, 16, 4096, 4096) == 0
    # few output tiles and a long K: fp32 partial sums of at least two slices
    for op in (mx.MX_OP_GEMM_BF16, mx.MX_OP_GEMM_MX):
        assert nv.mx_workspace_size(op, 128, 256, 12288) >= 2 * 128 * 256 * 4
    assert nv.mx_workspace_size(mx.MX_OP_MOE, 3 * 2, 96, 64) >= 3 * 2 * 64 * 4 + 3 * 2 * 4 + 3 * 4
    for bad in ((0, -1, 1, 1), (0, 1 << 40, 1, 1), (99, 1, 1, 1), (mx.MX_OP_MOE, 64 * 16 + 1, 64, 64)):
        assert nv.mx_workspace_size(*bad) == 0


def test_quantize_refusals(nv):
    q = nv.lib.mxfp4_quantize
    t = _mx(nv, 4, 64)

    def call(x=P(FAKE), dt=1, ld=64, sc=None, out=t, flags=None):
        return q(x, dt, ld, sc, None if out is None else ctypes.byref(out), flags, None)
    assert call(dt=9) == 4
    assert call(out=None) == 1 and call(x=None) == 1
    assert call(out=_mx(nv, 4, 48), ld=48) == 2 and call(out=_mx(nv, -1, 64)) == 2 and call(ld=32) == 2
    assert call(out=_mx(nv, 1 << 40, 64)) == 2
    assert call(out=_mx(nv, 4, 64, codes=None)) == 1 and call(out=_mx(nv, 4, 64, scales=None)) == 1
    assert call(x=P(FAKE + 4)) == 3 and call(ld=68) == 3 and call(out=_mx(nv, 4, 64, codes=FAKE + 8)) == 3
    assert call(out=_mx(nv, 4, 64, scales=FAKE + 2)) == 3 and call(flags=P(FAKE + 2)) == 3
    assert call(sc=P(FAKE)) == 6 and call(dt=3, sc=P(FAKE + 1)) == 3


def test_dequantize_refusals(nv):
    d = nv.lib.mxfp4_dequantize
    t = _mx(nv, 4, 64)
    assert d(None, P(FAKE), 1, 64, None) == 1 and d(ctypes.byref(t), None, 1, 64, None) == 1
    assert d(ctypes.byref(t), P(FAKE), 2, 64, None) == 4 and d(ctypes.byref(t), P(FAKE), 3, 64, None) == 4
    assert d(ctypes.byref(t), P(FAKE), 1, 63, None) == 2 and d(ctypes.byref(t), P(FAKE), 1, 68, None) == 3


def test_gemm_refusals(nv):
    g = nv.lib.mxfp4_gemm
    w, a = _mx(nv, 64, 128), _mx(nv, 100, 128)

    def call(a16=P(FAKE), aq=None, m=100, lda=128, wt=w, c=P(FAKE), dt=0, ldc=64, ws=P(FAKE), wsb=1 << 20):
        return g(a16, None if aq is None else ctypes.byref(aq), m, lda, None if wt is None else ctypes.byref(wt), c,
                 dt, ldc, ws, wsb, None)
    assert call(a16=None) == 6 and call(aq=a) == 6                       # neither, both
    assert call(wt=None) == 1 and call(c=None) == 1
    assert call(dt=2) == 4 and call(dt=3) == 4                           # C: fp32 or bf16
    assert call(m=-1) == 2 and call(lda=96) == 2 and call(ldc=63) == 2
    assert call(a16=None, aq=_mx(nv, 99, 128)) == 2 and call(a16=None, aq=_mx(nv, 100, 160)) == 2
    assert call(wt=_mx(nv, 64, 120), lda=120) == 2
    assert call(wt=_mx(nv, 1, 1 << 23), lda=1 << 23, ldc=1) == 2         # K beyond the tile's range
    assert call(lda=(1 << 22) + 8) == 2                                  # rows of A too far apart for a tile
    assert call(lda=132) == 3 and call(c=P(FAKE + 2)) == 3 and call(dt=1, c=P(FAKE + 1)) == 3
    assert call(ws=P(FAKE + 8)) == 3


def test_moe_refusals(nv):
    f = nv.lib.mxfp4_moe
    E, H, I = 4, 64, 32
    ws = nv.mx_workspace_size(2, 3 * 2, H, I)

    def call(x=P(FAKE), t=3, ldx=H, lg=P(FAKE), ldt=0, ldl=E, e=E, k=2, rn=1, gu=_mx(nv, E * 2 * I, H),
             dn=_mx(nv, E * H, I), y=P(FAKE), yd=1, ldy=H, ids=None, wt=None, w=P(FAKE), wsb=ws):
        return f(x, t, ldx, lg, ldt, ldl, e, k, rn, None if gu is None else ctypes.byref(gu),
                 None if dn is None else ctypes.byref(dn), y, yd, ldy, ids, wt, w, wsb, None)
    assert call(ldt=2) == 4 and call(yd=3) == 4
    assert call(gu=None) == 1 and call(dn=None) == 1 and call(x=None) == 1 and call(lg=None) == 1 and call(y=None) == 1
    assert call(t=65) == 2 and call(t=-1) == 2 and call(e=513) == 2 and call(e=0) == 2 and call(k=17) == 2
    assert call(k=0) == 6 and call(k=5) == 6 and call(rn=2) == 6
    assert call(gu=_mx(nv, E * 2 * I - 1, H)) == 2 and call(dn=_mx(nv, E * H + 1, I)) == 2
    assert call(gu=_mx(nv, 0, H), dn=_mx(nv, E * H, 0)) == 2
    assert call(ldx=32) == 2 and call(ldl=3) == 2 and call(ldy=63) == 2
    assert call(ldx=68) == 3 and call(lg=P(FAKE + 2)) == 3 and call(y=P(FAKE + 1)) == 3
    assert call(ids=P(FAKE + 2)) == 3 and call(wt=P(FAKE + 1)) == 3 and call(w=P(FAKE + 8)) == 3
    assert call(w=None) == 5 and call(wsb=ws - 1) == 5


def test_valid_calls_without_gpu_report_device(nv):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    t, w = _mx(nv, 4, 64), _mx(nv, 8, 64)
    assert nv.lib.mxfp4_quantize(P(FAKE), 1, 64, None, ctypes.byref(t), None, None) == 7
    assert nv.lib.mxfp4_dequantize(ctypes.byref(t), P(FAKE), 1, 64, None) == 7
    assert nv.lib.mxfp4_gemm(None, ctypes.byref(t), 4, 0, ctypes.byref(w), P(FAKE), 0, 8, None, 0, None) == 7


def test_reference_decodes_and_rounds_to_nearest():
    rng = np.random.default_rng(1)
    v = rng.standard_normal((40, 96)) * np.exp2(rng.integers(-40, 40, (40, 1)))
    codes, scales = mx_ref.quantize(v)
    back = mx_ref.dequantize(codes, scales)
    s = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    grid = np.concatenate((-mx_ref.E2M1, mx_ref.E2M1))
    best = np.abs((v / s)[..., None] - grid).min(axis=-1)
    assert np.allclose(np.abs(v - back) / s, best, rtol=0, atol=1e-12)
    amax = np.abs(v).reshape(40, 3, 32).max(axis=2)
    ratio = amax / np.ldexp(1.0, scales.astype(int) - 127)
    assert (ratio >= 4).all() and (ratio < 8).all()


def test_reference_ties_signs_and_edges():
    row = np.zeros(32)
    row[:14] = [4, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 7.9, -0.0, -0.25, -5, 0, 6]
    codes, scales = mx_ref.quantize(row[None])
    assert scales[0, 0] == 127
    nib = np.stack((codes[0] & 15, codes[0] >> 4), axis=1).reshape(-1)
    assert list(nib[:14]) == [6, 0, 2, 2, 4, 4, 6, 6, 7, 8, 8, 14, 0, 7]
    for bad in (np.nan, np.inf, -np.inf):
        r = row.copy()
        r[5] = bad
        c, s = mx_ref.quantize(r[None])
        assert s[0, 0] == 255 and not c.any() and np.isnan(mx_ref.dequantize(c, s)).all()
    c, s = mx_ref.quantize(np.full((1, 32), 2.0 ** -149))  # below the smallest scale's grid
    assert s[0, 0] == 0 and not c.any()


def test_reference_routing_masks_and_ties():
    ninf = -np.inf
    lg = np.array([[1.0, 1.0, 0.0, 1.0], [ninf, 2.0, ninf, ninf], [ninf] * 4, [0, np.nan, 1, 2], [0, np.inf, 1, 2]])
    ids, w = mx_ref.route(lg, 2, True)
    assert ids.tolist() == [[0, 1], [1, -1], [-1, -1], [-1, -1], [-1, -1]]
    assert np.allclose(w[0], 0.5) and w[1].tolist() == [1.0, 0.0] and not w[2:].any()
    assert np.isclose(mx_ref.route(lg, 2, False)[1][0].sum(), 2 * np.e / (3 * np.e + 1))


def test_binding_refusals(nv):
    import torch
    with pytest.raises(AssertionError):
        nv.MXFP4Tensor.empty(4, 48, "cpu")
    t = nv.MXFP4Tensor(torch.zeros((4, 32), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.uint8))
    with pytest.raises(AssertionError):
        t.c()  # 64 columns need two scale bytes per row (and a device tensor)
    with pytest.raises(AssertionError):
        nv.mx_quantize(torch.zeros((4, 64)))  # host tensor
    from bit_gemm_nvfp4_amd import mx
    with pytest.raises(AssertionError):
        mx._nbytes(torch.zeros(1, dtype=torch.uint8).expand(4096))  # a workspace that is not what it seems
    with pytest.raises(AssertionError):
        nv.mx_gemm(torch.zeros((4, 64)), t)  # fp32 activations
