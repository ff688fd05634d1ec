"""The MXFP4 expert layer on the GPU: the range and precision of what it carries between its products, and the
sizes that reach its forms."""
import numpy as np
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


@pytest.mark.parametrize("t, e, i", [(1, 1, 32), (3, 8, 96), (11, 2, 544), (64, 5, 160), (64, 300, 32)])
def test_inner_values_keep_the_bits_of_fp32(nv, t, e, i):
    # gate g of 8 bits (silu(g) = g from g = 104 on) and up b + c 2^-8 of 16 bits: the inner value g (b + c 2^-8) has
    # 24 bits, exact in fp32, and each output element is one of them
    h = 64
    rng = np.random.default_rng(t + i)
    gu, dn = _zeros(nv, e * 2 * i, h), _zeros(nv, e * h, i)

    def put(w, row, col, code):
        w.codes[row, col // 2] |= code << (4 * (col % 2))
    for r in range(i):
        rows = torch.arange(e, device=DEV) * 2 * i + r
        put(gu, rows, r % 16, 2)
        put(gu, rows + i, 16 + r * 5 % 16, 2)
        put(gu, rows + i, 32 + r * 3 % 16, 2)
    pick = np.array([o * 7 % i for o in range(h)])
    for o in range(h):
        put(dn, torch.arange(e, device=DEV) * h + o, int(pick[o]), 2 + 8 * (o % 2))
    xd = np.zeros((t, h))
    xd[:, :32] = rng.integers(128, 256, (t, 32))
    xd[:, 32:48] = rng.integers(128, 256, (t, 16)) / 256
    x = torch.from_numpy(xd).to(torch.bfloat16).to(DEV)
    logits = torch.from_numpy(rng.standard_normal((t, e)).astype(np.float32)).to(DEV)
    r = np.arange(i)
    inner = xd[:, r % 16] * (xd[:, 16 + r * 5 % 16] + xd[:, 32 + r * 3 % 16])
    want = inner[:, pick] * np.where(np.arange(h) % 2, -1, 1)
    y = nv.mx_moe(x, logits, gu, dn, 1, dtype=torch.float32)
    assert np.array_equal(y.double().cpu().numpy(), want)
