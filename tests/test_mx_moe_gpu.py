"""The MXFP4 expert layer on the GPU: the range and precision of what it carries between its products, and the
sizes that reach its forms."""
import numpy as np
import pytest
import torch

import mx_ref
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


# (tokens, experts, top_k, H, I, 16-row tiles per workgroup of the first product on 256 CUs): all with a last run shorter
# than the others.  H below and above eight groups of 512 columns, with a rest; more than sixteen tokens on one expert;
# slots that are experts and slots that are choices; the second product in its two forms.
RUNS = [(40, 8, 1, 4064, 1504, 3), (12, 8, 1, 4064, 2272, 5), (64, 8, 2, 4064, 2272, 5), (40, 8, 1, 4064, 6176, 12),
        (3, 16, 2, 4064, 1984, 3), (40, 8, 1, 4640, 1504, 3), (64, 8, 2, 4640, 2272, 5), (33, 8, 1, 4640, 6176, 12),
        (5, 32, 2, 4640, 4544, 12)]


def _values(w, rows):
    """float64 values of rows of an MXFP4 tensor."""
    table = torch.tensor([*mx_ref.E2M1, *-mx_ref.E2M1], dtype=torch.float64, device=DEV)
    c = w.codes[rows]
    v = torch.stack((table[(c & 15).int()], table[(c >> 4).int()]), dim=2).view(c.shape[0], -1, 32)
    return (v * torch.exp2(w.scales[rows].double() - 127).unsqueeze(2)).view(c.shape[0], -1)


def _sparse(rows, cols, col, code):
    """Codes with `code` at column col[n][row] of each row, for each n."""
    c = torch.zeros((rows, cols // 2), dtype=torch.int32, device=DEV)
    r = torch.arange(rows, device=DEV)
    for n in range(len(col)):
        c[r, col[n] // 2] |= code[n] << (4 * (col[n] % 2))
    return c.to(torch.uint8)


@pytest.mark.parametrize("dense", ["up", "down"])
@pytest.mark.parametrize("case", RUNS, ids=lambda c: "x".join(map(str, c)))
def test_runs_of_tiles_are_exact(nv, case, dense):
    # All values are small multiples of a power of two and silu(g) = g from g = 104 on, so every sum is exact in fp32 and
    # the outputs are the float64 ones.  "up": the first product's operands are dense and the second picks inner
    # values; "down": the first makes small inner values and the second's weights are dense.
    t, e, k, h, i, run = case
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    slots = t * k if t * k < e else e
    assert run == min(12, max(1, -(-slots * (i // 16) // cus))) and (i // 16) % run, "not the run this case is for"
    g = torch.Generator(device=DEV)
    g.manual_seed(h + i + t)

    def rand(lo, hi, shape):
        return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)
    ngu, ndn = e * 2 * i, e * h
    if dense == "up":
        x = rand(0, 2, (t, h))
        codes = rand(0, 4, (ngu, h))  # 0 to 1.5
        codes.view(e, 2, i, h)[:, 1] += 8 * rand(0, 2, (e, i, h))
        gu = nv.MXFP4Tensor((codes[:, ::2] | codes[:, 1::2] << 4).to(torch.uint8), rand(126, 128, (ngu, h // 32)).to(torch.uint8))
        del codes
        row = torch.arange(ndn, device=DEV)
        col = [row % h % i, (row % h + h) % i]  # of every inner value, one or two go into an output
        code = [2 + 8 * rand(0, 2, (ndn,)), 2 + 8 * rand(0, 2, (ndn,))]
        if i <= h:
            col, code = col[:1], code[:1]
        dn = nv.MXFP4Tensor(_sparse(ndn, i, col, code), torch.full((ndn, i // 32), 127, dtype=torch.uint8, device=DEV))
    else:
        x = rand(1, 4, (t, h))
        x[:, 0] = 128
        row = torch.arange(ngu, device=DEV)
        up = row // i % 2 == 1
        col = torch.where(up, 1 + (row % i * 37 + row // (2 * i)) % (h - 1), torch.zeros_like(row))
        code = torch.where(up, rand(1, 6, (ngu,)) + 8 * rand(0, 2, (ngu,)), torch.full_like(row, 2, dtype=torch.int32))
        gu = nv.MXFP4Tensor(_sparse(ngu, h, [col], [code]), torch.full((ngu, h // 32), 127, dtype=torch.uint8, device=DEV))
        dn = nv.MXFP4Tensor(rand(0, 256, (ndn, i // 2)).to(torch.uint8), rand(125, 129, (ndn, i // 32)).to(torch.uint8))
    # the chosen experts of a row have the same logit: weights 1 / k.  Up to 24 rows choose expert e / 2.
    logits = torch.rand((t, e), generator=g, device=DEV) - 2
    first = torch.where(torch.arange(t, device=DEV) % 5 < 3, torch.full((t,), e // 2, device=DEV), torch.arange(t, device=DEV) % e)
    for c in range(k):
        logits[torch.arange(t, device=DEV), (first + 3 * c) % e] = 1
    y = nv.mx_moe(x.to(torch.bfloat16), logits, gu, dn, k, dtype=torch.float32).double()

    xd, want, mag = x.double(), torch.zeros((t, h), dtype=torch.float64, device=DEV), torch.zeros((t, h), dtype=torch.float64, device=DEV)
    unit = 2.0 ** -4 if dense == "up" else 2.0 ** 3  # every product is a multiple of it
    for j in range(e):
        rows = (logits[:, j] == 1).nonzero().flatten()
        if len(rows) == 0:
            continue
        w = _values(gu, slice(j * 2 * i, (j + 1) * 2 * i))
        gate, upv = xd[rows] @ w[:i].t(), xd[rows] @ w[i:].t()
        assert float(gate.min()) >= 104
        inner = gate * upv
        assert float((inner / unit).abs().max()) < 2 ** 24
        w = _values(dn, slice(j * h, (j + 1) * h))
        want[rows] += inner @ w.t()
        mag[rows] += inner.abs() @ w.abs().t()
    assert float(mag.max()) / unit < 2 ** 24  # nothing is rounded on the way
    wrong = (y != want / k).nonzero()
    assert len(wrong) == 0, (len(wrong), wrong[:4].tolist())
