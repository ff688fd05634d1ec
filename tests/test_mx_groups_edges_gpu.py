"""Grouped products, router, weighted sum and expert layer at sizes and arguments that their other tests leave out."""
import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def test_an_mxfp4_output_keeps_no_earlier_flags(nv):
    g = gen(1)
    x = randn(g, 40, 64)
    x[3, 5] = float("nan")
    flags = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = nv.mx_quantize(x, flags=flags)
    assert q.flags is flags and int(flags) == 1
    a, w = randn(g, 40, 96).to(torch.bfloat16), nv.mx_quantize(randn(g, 128, 96) * 0.1)
    nv.mx_grouped_gemm(a, w, torch.tensor([0, 40], dtype=torch.int32, device=DEV), swiglu=True, out=q)
    assert q.flags is None and bool(nv.mx_dequantize(q).isfinite().all())
