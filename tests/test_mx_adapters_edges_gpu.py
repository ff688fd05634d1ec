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


# More than 1024 rows take other forms of A . V^T, by rank: up to 16, up to 32, above; tiles of ranks, rows and columns of K that
# end inside one; adapters in order (up to 511 of them), one, and too many to be sorted.
@pytest.mark.parametrize("act", ["bf16", "mx"])
@pytest.mark.parametrize("count", [1, 7, 600])
@pytest.mark.parametrize("m, n, k, rank", [(1025, 50, 96, 8), (1300, 130, 1056, 16), (1025, 64, 544, 24), (1300, 33, 160, 32), (1056, 70, 4128, 40),
                                           (1300, 100, 32, 72), (1025, 40, 1056, 136), (2100, 300, 608, 64), (1200, 48, 96, 256)])
def test_more_than_1024_rows(nv, m, n, k, rank, count, act):
    print(m, n, k, rank, count, act, flush=True)
    a, w, down, up, scales, index = case(nv, m + k, m, n, k, rank, count)
    a_q = nv.mx_quantize(a) if act == "mx" else None
    want, err = expected(nv, a, w, down, up, scales, index, a_q)
    check(nv.mx_gemm_adapters(a, w, down, up, index, scales=scales, a_q=a_q), want, err, torch.float32)


@pytest.mark.parametrize("m, rank", [(700, 24), (1300, 16), (1300, 40)])
def test_rows_of_one_request_after_the_other_with_many_adapters(nv, m, rank):
    a, w, down, up, scales, index = case(nv, m, m, 96, 544, rank, 600)
    index[:] = torch.arange(m, device=DEV).to(torch.int32) // 90 * 37 - 1  # runs that end inside tiles, the first of none
    want, err = expected(nv, a, w, down, up, scales, index)
    check(nv.mx_gemm_adapters(a, w, down, up, index, scales=scales), want, err, torch.float32)
