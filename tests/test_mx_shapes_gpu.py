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
