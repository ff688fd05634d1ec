"""The MXFP4 expert layer on the GPU: the range and precision of what it carries between its products, and the
sizes that reach its forms."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


def _zeros(nv, rows, cols, scale=127):
    return nv.MXFP4Tensor(torch.zeros((rows, cols // 2), dtype=torch.uint8, device=DEV),
                          torch.full((rows, cols // 32), scale, dtype=torch.uint8, device=DEV))


def _one_inner_value(nv, t, e, gate, up, down_scale=127):
    """A layer of 32 x 32 whose inner element 0 is silu(gate) * up in every token (x[0] = gate, x[1] = up) and goes
    out with weight 1 (element 0), -1 (element 1) and 0 (the others)."""
    gu, dn = _zeros(nv, e * 64, 32), _zeros(nv, e * 32, 32, down_scale)
    gu.codes.view(e, 64, 16)[:, 0, 0] = 0x02
    gu.codes.view(e, 64, 16)[:, 32, 0] = 0x20
    dn.codes.view(e, 32, 16)[:, 0, 0] = 0x02
    dn.codes.view(e, 32, 16)[:, 1, 0] = 0x0A
    x = torch.zeros((t, 32), dtype=torch.bfloat16, device=DEV)
    x[:, 0], x[:, 1] = gate, up
    assert float(x[0, 0]) == gate and float(x[0, 1]) == up
    return x, gu, dn


# one token per expert, and the form for several
@pytest.mark.parametrize("t, e", [(1, 1), (2, 8), (40, 2)])
@pytest.mark.parametrize("sign", [1, -1])
def test_inner_values_beyond_bf16_stay_finite(nv, t, e, sign):
    # 33 * 2^59 * 31 * 2^59 = 1023 * 2^118 is finite in fp32 but rounds to infinity in bf16
    x, gu, dn = _one_inner_value(nv, t, e, 33 * 2.0 ** 59, sign * 31 * 2.0 ** 59, 127 - 120)
    logits = torch.zeros((t, e), device=DEV)
    y = nv.mx_moe(x, logits, gu, dn, 1, dtype=torch.float32)
    want = torch.zeros((t, 32), device=DEV)
    want[:, 0], want[:, 1] = sign * 1023 / 4, -sign * 1023 / 4
    assert torch.equal(y, want)


@pytest.mark.parametrize("t, e", [(1, 1), (2, 8), (40, 2)])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_inner_values_go_out_as_in_fp32(nv, t, e, sign):
    x, gu, dn = _one_inner_value(nv, t, e, 2.0 ** 70, sign * 2.0 ** 70)
    y = nv.mx_moe(x, torch.zeros((t, e), device=DEV), gu, dn, 1, dtype=torch.float32)
    inf = float("inf") * sign
    assert bool((y[:, 0] == inf).all()) and bool((y[:, 1] == -inf).all())
    assert bool(torch.isnan(y[:, 2:]).all())  # infinity times zero
