"""Adapters beside an MXFP4 projection at sizes that their other tests leave out, against the plain float64 form."""
import pytest
import torch

from gpu_util import DEV
from test_mx_adapters_gpu import case, check, expected, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


@pytest.mark.parametrize("m", [2, 40, 200])
def test_an_up_matrix_of_more_than_two_billion_elements(nv, m):
    n, k, rank, count = 1 << 23, 32, 256, 2
    g = gen(m)
    w = nv.MXFP4Tensor(torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8),
                       torch.full((n, 1), 122, device=DEV, dtype=torch.uint8))
    a = torch.randn((m, k), generator=g, device=DEV).to(torch.bfloat16)
    down = (torch.randn((count, rank, k), generator=g, device=DEV) * 0.2).to(torch.bfloat16)
    up = torch.empty((count, n, rank), dtype=torch.bfloat16, device=DEV)
    for part in up.view(-1).split(1 << 28):
        part.normal_(generator=g)
    index = torch.arange(m, device=DEV).to(torch.int32) % 3  # the third: none
    got = nv.mx_gemm_adapters(a, w, down, up, index, dtype=torch.bfloat16)
    # (parts whose scale bytes start 16-byte aligned)
    for lo, hi in ((0, 304), (n // 2 - 96, n // 2 + 96), (n - 304, n)):
        part = nv.MXFP4Tensor(w.codes[lo:hi], w.scales[lo:hi])
        want, err = expected(nv, a, part, down, up[:, lo:hi], None, index)
        check(got[:, lo:hi], want, err, torch.bfloat16)
