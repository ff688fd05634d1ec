"""Router, grouped products, weighted sum and expert layer on the CPU: refusals before anything touches the GPU, and
workspace sizes."""
import ctypes

import pytest

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first
P = ctypes.c_void_p
MAX_ROWS = 1 << 24


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


def _mx(rows, cols, codes=FAKE, scales=FAKE):
    from bit_gemm_nvfp4_amd.mx import CMXTensor
    return CMXTensor(codes, scales, rows, cols)


def _ref(t):
    return None if t is None else ctypes.byref(t)


def _gpu():
    import torch
    return torch.cuda.is_available()


def test_workspace_sizes(nv):
    from bit_gemm_nvfp4_amd import mx
    assert mx.ROUTE_ONE_LAUNCH == 16 and nv.mx_workspace_size(mx.MX_OP_ROUTE, 16, 8, 512) == 0  # one workgroup
    assert nv.mx_workspace_size(mx.MX_OP_ROUTE, 17, 8, 512) == 2 * 512 * 4  # a table of counts: 16 rows a workgroup,
    assert nv.mx_workspace_size(mx.MX_OP_ROUTE, 1 << 20, 16, 512) == 256 * 512 * 4  # never more than 256
    assert nv.mx_workspace_size(mx.MX_OP_GROUP_ROWS, 4096, 1, 40) == 0
    assert nv.mx_workspace_size(mx.MX_OP_GROUP_ROWS, 4097, 1, 40) == 2 * 40 * 4
    for bad in ((mx.MX_OP_ROUTE, MAX_ROWS, 2, 8), (mx.MX_OP_ROUTE, 100, 2, 513), (mx.MX_OP_GROUP_ROWS, -1, 2, 8)):
        assert nv.mx_workspace_size(*bad) == 0
    size = nv.lib.mxfp4_experts_workspace_size
    assert size(0, 8, 2, 64, 32, 1, 1) == 0
    # at least the inner activations and the experts' outputs
    assert size(100, 8, 2, 64, 32, 0, 0) >= 200 * 32 * 2 + 200 * 64 * 4
    assert size(100, 8, 2, 64, 32, 1, 1) >= 100 * 34 + 200 * 17 + 200 * 64 * 2
    for bad in ((100, 8, 0, 64, 32, 1, 1), (MAX_ROWS, 8, 2, 64, 32, 1, 1), (100, 0, 2, 64, 32, 1, 1), (100, 513, 2, 64, 32, 1, 1),
                (100, 8, 2, 1 << 21, 32, 1, 1), (100, 8, 2, 64, 32, 1, 2), (-1, 8, 2, 64, 32, 1, 1)):
        assert size(*bad) == 0


def test_route_refusals(nv):
    ws = nv.mx_workspace_size(3, 100, 2, 8)
    assert ws > 0

    def call(lg=P(FAKE), dt=0, t=100, ld=8, e=8, k=2, rn=1, ids=P(FAKE), wt=P(FAKE), off=P(FAKE), rows=P(FAKE), pl=P(FAKE),
             w=P(FAKE), wsb=ws):
        return nv.lib.mxfp4_route(lg, dt, t, ld, e, k, rn, ids, wt, off, rows, pl, w, wsb, None)
    assert call(dt=2) == 4 and call(dt=3) == 4
    assert call(t=-1) == 2 and call(e=0) == 2 and call(e=513, ld=513) == 2 and call(k=17) == 2 and call(t=MAX_ROWS) == 2 and call(ld=7) == 2
    assert call(k=0) == 6 and call(k=9) == 6 and call(rn=2) == 6
    for name in ("lg", "ids", "wt", "off", "rows", "pl"):
        assert call(**{name: None}) == 1
        assert call(**{name: P(FAKE + 2)}) == 3
    assert call(w=P(FAKE + 8)) == 3 and call(w=None) == 5 and call(wsb=ws - 1) == 5
    if not _gpu():
        assert call() == 7 and call(t=16, w=None) == 7 and call(t=0, lg=None, ids=None, wt=None, rows=None, pl=None, w=None) == 7


def test_group_rows_refusals(nv):
    ws = nv.mx_workspace_size(4, 5000, 2, 8)

    def call(ids=P(FAKE), t=5000, k=2, g=8, off=P(FAKE), rows=P(FAKE), pl=None, w=P(FAKE), wsb=ws):
        return nv.lib.mxfp4_group_rows(ids, t, k, g, off, rows, pl, w, wsb, None)
    assert call(t=-1) == 2 and call(g=0) == 2 and call(g=513) == 2 and call(t=MAX_ROWS) == 2 and call(k=0) == 6
    assert call(ids=None) == 1 and call(off=None) == 1 and call(rows=None) == 1
    assert call(ids=P(FAKE + 1)) == 3 and call(off=P(FAKE + 2)) == 3 and call(rows=P(FAKE + 2)) == 3 and call(pl=P(FAKE + 2)) == 3
    assert call(w=P(FAKE + 4)) == 3 and call(w=None) == 5 and call(wsb=ws - 1) == 5
    if not _gpu():
        assert call() == 7 and call(t=100, w=None) == 7


def test_grouped_gemm_refusals(nv):
    w, a = _mx(4 * 64, 128), _mx(100, 128)

    def call(a16=P(FAKE), aq=None, ar=100, lda=128, mp=None, off=P(FAKE), g=4, rows=100, wt=w, sw=0, c=P(FAKE), dt=0, ldc=64, cq=None):
        return nv.lib.mxfp4_grouped_gemm(a16, _ref(aq), ar, lda, mp, off, g, rows, _ref(wt), sw, c, dt, ldc, _ref(cq), None)
    assert call(a16=None) == 6 and call(aq=a) == 6                       # neither, both
    assert call(c=None, cq=_mx(100, 64)) == 6 and call(sw=2) == 6        # an MXFP4 C without swiglu
    assert call(sw=1, cq=_mx(100, 32)) == 6
    assert call(wt=None) == 1 and call(c=None) == 1 and call(off=None) == 1
    assert call(dt=2) == 4
    assert call(rows=-1, ar=-1) == 2 and call(g=0) == 2 and call(g=513) == 2 and call(g=3) == 2 and call(rows=99) == 2
    assert call(rows=MAX_ROWS + 1, ar=MAX_ROWS + 1) == 2 and call(mp=P(FAKE), ar=MAX_ROWS + 1) == 2
    assert call(wt=_mx(256, 0), lda=0) == 2 and call(wt=_mx(4, 1 << 21), lda=1 << 21, ldc=1) == 2
    assert call(lda=(1 << 20) + 8) == 2 and call(lda=96) == 2 and call(ldc=63) == 2
    assert call(wt=_mx(4 * 63, 128), sw=1, ldc=63) == 2                  # halves of 31.5 rows
    assert call(g=1, wt=_mx((1 << 24) + 1, 32), lda=32, ldc=1 << 25) == 2
    assert call(g=1, wt=_mx(1 << 12, 1 << 20), lda=1 << 20, sw=1, ldc=1 << 11) == 2   # 2^30 bytes of gate rows
    assert call(mp=P(FAKE), ar=1 << 23) == 2                             # picked from 2^31 bytes
    assert call(a16=None, aq=_mx(99, 128)) == 2 and call(a16=None, aq=_mx(100, 160)) == 2
    assert call(c=None, cq=_mx(100, 64), sw=1) == 2                      # N / 2 = 32 columns
    assert call(lda=132) == 3 and call(c=P(FAKE + 2)) == 3 and call(off=P(FAKE + 2)) == 3 and call(mp=P(FAKE + 1)) == 3
    if not _gpu():
        # (which tiles fit one launch is asked behind the device)
        assert call() == 7 and call(sw=1, c=None, cq=_mx(100, 32)) == 7 and call(mp=P(FAKE), ar=(1 << 23) - 1) == 7


def test_combine_refusals(nv):
    def call(z=P(FAKE), zt=1, zr=10, ldz=64, pl=P(FAKE), wt=P(FAKE), t=4, k=2, cols=64, y=P(FAKE), yt=1, ldy=64):
        return nv.lib.mxfp4_combine(z, zt, zr, ldz, pl, wt, t, k, cols, y, yt, ldy, None)
    assert call(zt=2) == 4 and call(yt=3) == 4
    assert call(t=-1) == 2 and call(zr=-1) == 2 and call(cols=65) == 2 and call(ldy=63) == 2 and call(t=MAX_ROWS) == 2
    assert call(k=0) == 6
    assert call(z=None) == 1 and call(pl=None) == 1 and call(wt=None) == 1 and call(y=None) == 1
    assert call(z=P(FAKE + 1)) == 3 and call(pl=P(FAKE + 2)) == 3 and call(wt=P(FAKE + 1)) == 3 and call(y=P(FAKE + 1)) == 3
    if not _gpu():
        assert call() == 7


def test_experts_refusals(nv):
    E, H, I = 4, 64, 32
    ws = nv.lib.mxfp4_experts_workspace_size(300, E, 2, H, I, 1, 1)

    def call(x=P(FAKE), t=300, ldx=H, lg=P(FAKE), ldt=0, ldl=E, e=E, k=2, rn=1, qa=1, gu=_mx(E * 2 * I, H), dn=_mx(E * H, I),
             y=P(FAKE), yd=1, ldy=H, ids=None, wt=None, w=P(FAKE), wsb=ws):
        return nv.lib.mxfp4_experts(x, t, ldx, lg, ldt, ldl, e, k, rn, qa, _ref(gu), _ref(dn), y, yd, ldy, ids, wt, w, wsb, None)
    assert call(ldt=2) == 4 and call(yd=3) == 4
    assert call(gu=None) == 1 and call(dn=None) == 1 and call(x=None) == 1 and call(lg=None) == 1 and call(y=None) == 1
    assert call(t=-1) == 2 and call(e=513) == 2 and call(e=0) == 2 and call(k=17) == 2 and call(t=MAX_ROWS) == 2
    assert call(k=0) == 6 and call(k=5) == 6 and call(rn=2) == 6 and call(qa=2) == 6
    assert call(gu=_mx(E * 2 * I - 1, H)) == 2 and call(dn=_mx(E * H + 1, I)) == 2
    assert call(gu=_mx(0, H), dn=_mx(E * H, 0)) == 2
    assert call(t=1 << 22, k=1, ldx=1 << 10) == 2                        # x of 2^33 bytes
    assert call(ldx=32) == 2 and call(ldl=3) == 2 and call(ldy=63) == 2 and call(ldx=68) == 3
    assert call(lg=P(FAKE + 2)) == 3 and call(y=P(FAKE + 1)) == 3 and call(ids=P(FAKE + 2)) == 3 and call(wt=P(FAKE + 1)) == 3
    assert call(w=P(FAKE + 8)) == 3 and call(w=None) == 5 and call(wsb=ws - 1) == 5
    if not _gpu():
        assert call() == 7


def test_binding_refusals(nv):
    import torch
    from bit_gemm_nvfp4_amd import mx
    cpu = torch.device("cpu")
    t = torch.zeros((3, 2), dtype=torch.int32)
    assert mx._words(t, "t", cpu, torch.int32, 3, 2) == t.data_ptr()
    for bad in (t.long(), t[:2], t.t(), t.view(-1)):
        with pytest.raises(AssertionError):
            mx._words(bad, "t", cpu, torch.int32, 3, 2)
    with pytest.raises(AssertionError):
        nv.mx_route(torch.zeros((4, 8)), 2)  # host tensor
    with pytest.raises(AssertionError):
        nv.mx_group_rows(t, 4)
    with pytest.raises(AssertionError):
        nv.mx_grouped_gemm(torch.zeros((4, 64)), t, t)


def test_adapters_refusals(nv):
    size = nv.lib.mxfp4_adapters_workspace_size
    M, N, K, R, C = 100, 64, 128, 16, 3
    ws = size(M, N, K, C, R, 0)
    assert ws >= M * R * 6 + M * 4 and size(16, N, K, C, R, 0) >= 16 * R * 4 and size(M, N, K, 0, R, 0) == 0  # T; the rows' order
    assert size(0, N, K, C, R, 0) == 0 and size(M, N, K, C, 12, 0) == 0 and size(MAX_ROWS + 1, N, K, C, R, 0) == 0

    def call(a16=P(FAKE), aq=None, m=M, lda=K, wt=_mx(N, K), idx=P(FAKE), cnt=C, r=R, dn=P(FAKE), up=P(FAKE), sc=None, c=P(FAKE), dt=0,
             ldc=N, w=P(FAKE), wsb=ws):
        return nv.lib.mxfp4_gemm_adapters(a16, _ref(aq), m, lda, _ref(wt), idx, cnt, r, dn, up, sc, c, dt, ldc, w, wsb, None)
    assert call(wt=None) == 1 and call(a16=None) == 1 and call(a16=None, aq=_mx(M, K)) == 1   # the branch takes bf16
    assert call(idx=None) == 1 and call(dn=None) == 1 and call(up=None) == 1 and call(c=None) == 1
    assert call(dt=2) == 4
    assert call(m=-1) == 2 and call(m=MAX_ROWS + 1) == 2 and call(lda=96) == 2 and call(ldc=63) == 2 and call(cnt=-1) == 2
    assert call(cnt=(1 << 16) + 1) == 2 and call(lda=(1 << 21) + 8) == 2
    for rank in (0, 4, 12, 264):
        assert call(r=rank) == 2
    assert call(aq=_mx(M - 1, K)) == 2 and call(aq=_mx(M, K + 32)) == 2
    assert call(lda=132) == 3 and call(dn=P(FAKE + 8)) == 3 and call(up=P(FAKE + 8)) == 3 and call(idx=P(FAKE + 2)) == 3
    assert call(sc=P(FAKE + 2)) == 3 and call(c=P(FAKE + 2)) == 3 and call(w=P(FAKE + 8)) == 3
    need = size(M, N, 32, C, R, 0)
    assert call(w=None) == 5 and call(wsb=need - 1) == 5
    if not _gpu():
        assert call() == 7 and call(wsb=need) == 7 and call(cnt=0, dn=None, up=None, w=None) == 7 and call(aq=_mx(M, K)) == 7
