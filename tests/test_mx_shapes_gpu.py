"""The MXFP4 products on the GPU at the sizes that reach their tile shapes and limits."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


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
