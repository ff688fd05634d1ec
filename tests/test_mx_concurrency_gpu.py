"""The MXFP4 entry points called from several host threads at a time, each on a stream of its own."""
import threading

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


def test_threads_on_their_own_streams():
    import bit_gemm_nvfp4_amd as nv
    g = torch.Generator(device=DEV)
    g.manual_seed(5)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=DEV)
    t, e, k, h, i = 12, 6, 2, 128, 96
    gu, dn = nv.mx_quantize(randn(e * 2 * i, h)), nv.mx_quantize(randn(e * h, i))
    w, wl = nv.mx_quantize(randn(h, h)), nv.mx_quantize(randn(200, 12288))
    inputs = [(randn(t, h).to(torch.bfloat16), randn(t, e), randn(40, 12288).to(torch.bfloat16)) for _ in range(4)]

    def chain(x, logits, big):
        y = nv.mx_moe(nv.mx_gemm(nv.mx_quantize(x), w, dtype=torch.bfloat16), logits, gu, dn, k)
        return y, nv.mx_gemm(big, wl), nv.mx_gemm(nv.mx_quantize(big), wl), nv.mx_dequantize(nv.mx_quantize(y))
    want = [chain(*args) for args in inputs]
    torch.cuda.synchronize()
    got, errors = [[] for _ in inputs], []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    got[n].append(chain(*inputs[n]))
        except Exception as err:  # noqa: BLE001 - reported by the test's own thread
            errors.append(err)
    threads = [threading.Thread(target=work, args=(n,)) for n in range(len(inputs))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for n, outs in enumerate(got):
        assert len(outs) == 20
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want[n]))
