"""Router, grouped products, expert layer and adapters as a program uses them: together, captured and replayed, from several
host threads, on other streams, with kept workspaces, and past 2^31 bytes."""
import threading

import pytest
import torch

from gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nv():
    import bit_gemm_nvfp4_amd as m
    return m


class Layer:
    """A projection with adapters, then experts, then the projection back with the same adapters' second set."""

    def __init__(self, nv, seed, h=256, e=10, i=96, k=3, adapters=6, rank=16):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device=DEV)
        self.nv, self.h, self.e, self.k, self.adapters = nv, h, e, k, adapters
        self.w_in, self.w_out = nv.mx_quantize(randn(h, h) * 0.06), nv.mx_quantize(randn(h, h) * 0.06)
        self.router = (randn(e, h) * 0.06).to(torch.bfloat16)
        self.gu, self.dn = nv.mx_quantize(randn(e * 2 * i, h) * 0.06), nv.mx_quantize(randn(e * h, i) * 0.1)
        self.down = [(randn(adapters, rank, h) * 0.06).to(torch.bfloat16) for _ in range(2)]
        self.up = [(randn(adapters, h, rank) * 0.2).to(torch.bfloat16) for _ in range(2)]
        self.scales = torch.rand(adapters, generator=g, device=DEV)

    def inputs(self, seed, t):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        x = torch.randn((t, self.h), generator=g, device=DEV).to(torch.bfloat16)
        index = torch.randint(-1, self.adapters, (t,), generator=g, device=DEV).to(torch.int32)
        return x, index

    def __call__(self, x, index, quantize_acts=True):
        nv = self.nv
        a_q = nv.mx_quantize(x) if quantize_acts else None
        y = nv.mx_gemm_adapters(x, self.w_in, self.down[0], self.up[0], index, scales=self.scales, a_q=a_q, dtype=torch.bfloat16)
        logits = nv.mx_gemm(y, nv.mx_quantize(self.router), dtype=torch.float32)
        z, ids, wts = nv.mx_experts(y, logits, self.gu, self.dn, self.k, quantize_acts=quantize_acts, routing=True)
        out = nv.mx_gemm_adapters(z, self.w_out, self.down[1], self.up[1], index, dtype=torch.float32)
        return out, z, ids, wts


@pytest.mark.parametrize("quantize_acts", [True, False])
@pytest.mark.parametrize("t", [1, 16, 33, 300])
def test_captured_and_replayed(nv, t, quantize_acts):
    print(t, quantize_acts, flush=True)
    layer = Layer(nv, 1)
    x, index = layer.inputs(2, t)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer(x, index, quantize_acts)
    torch.cuda.current_stream().wait_stream(stream)
    graphs, outs = [], []
    for _ in range(2):  # two graphs side by side
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer(x, index, quantize_acts))
        graphs.append(graph)
    for seed in range(4):
        nx, ni = layer.inputs(10 + seed, t)
        x.copy_(nx)
        index.copy_(ni)
        graphs[seed % 2].replay()
        got = [o.clone() for o in outs[seed % 2]]
        want = layer(nx, ni, quantize_acts)  # eager work between the replays
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_threads_on_their_own_streams(nv):
    layer = Layer(nv, 3)
    inputs = [layer.inputs(n, t) for n, t in enumerate((5, 40, 130, 700))]
    want = [layer(*args) for args in inputs]
    torch.cuda.synchronize()
    got, errors = [[] for _ in inputs], []

    def work(n):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got[n].append(layer(*inputs[n]))
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
        assert len(outs) == 10
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want[n]))


def test_kept_workspaces_need_no_contents(nv):
    t, e, k, h, i = 200, 8, 2, 128, 64
    layer = Layer(nv, 4, h=h, e=e, i=i, k=k)
    x, index = layer.inputs(1, t)
    logits = torch.randn((t, e), device=DEV)
    ws = nv.mx_experts_workspace(t, e, k, layer.gu, layer.dn)
    wa = nv.mx_adapters_workspace(t, layer.w_in, layer.adapters, 16)
    want = nv.mx_experts(x, logits, layer.gu, layer.dn, k), nv.mx_gemm_adapters(x, layer.w_in, layer.down[0], layer.up[0], index)
    for fill in (0, 0xFF, 0x7F):
        ws.fill_(fill)
        wa.fill_(fill)
        got = (nv.mx_experts(x, logits, layer.gu, layer.dn, k, workspace=ws),
               nv.mx_gemm_adapters(x, layer.w_in, layer.down[0], layer.up[0], index, workspace=wa))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(nv.NVFP4Error):
        nv.mx_experts(x, logits, layer.gu, layer.dn, k, workspace=ws[:-256])


def test_weights_past_two_gigabytes(nv):
    groups, n, k = 5, 1 << 17, 8192  # 2.7 GB of codes
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    codes = torch.randint(0, 256, (groups * n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(118, 124, (groups * n, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    w = nv.MXFP4Tensor(codes, scales)
    x = torch.randn((9, k), generator=g, device=DEV).to(torch.bfloat16)
    offsets = torch.tensor([0, 2, 2, 3, 5, 9], dtype=torch.int32, device=DEV)
    got = nv.mx_grouped_gemm(x, w, offsets)
    for lo, hi, j in ((0, 2, 0), (3, 5, 3), (5, 9, 4)):
        part = nv.MXFP4Tensor(codes[j * n:(j + 1) * n], scales[j * n:(j + 1) * n])
        want = nv.mx_gemm(x[lo:hi], part)
        mag = (x[lo:hi].float().abs().sum(1, keepdim=True) * 6 * 2.0 ** -4)
        # two fp32 sums of the same products, each within (K / 8 + 16) 2^-24 of the magnitudes
        assert bool(((got[lo:hi] - want).abs() <= 2 * (k / 8 + 16) * 2.0 ** -24 * mag).all())


def test_512_groups_and_adapters_beyond_the_sort(nv):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    groups, n, k = 512, 32, 64
    w = nv.mx_quantize(torch.randn((groups * n, k), generator=g, device=DEV))
    wd = nv.mx_dequantize(w, torch.float32).double().view(groups, n, k)
    ids = torch.randint(0, groups, (3000,), generator=g, device=DEV).to(torch.int32)
    ids[ids % 7 == 3] = 500
    r = nv.mx_group_rows(ids, groups)
    x = torch.randn((3000, k), generator=g, device=DEV).to(torch.bfloat16)
    got = nv.mx_grouped_gemm(x, w, r.offsets, rows=r.rows)[r.places.view(-1).long()]
    want, mag = torch.zeros((3000, n), dtype=torch.float64, device=DEV), torch.zeros((3000, n), dtype=torch.float64, device=DEV)
    for j in torch.unique(ids).tolist():
        rows = (ids == j).nonzero().flatten()
        want[rows], mag[rows] = x[rows].double() @ wd[j].t(), x[rows].double().abs() @ wd[j].abs().t()
    assert bool(((got.double() - want).abs() <= (k / 8 + 16) * 2.0 ** -24 * mag + 2.0 ** -23 * want.abs()).all())
    # more adapters than the sort has groups: the rows stay in their order
    count, rank, m = 600, 8, 150
    down = torch.randn((count, rank, k), generator=g, device=DEV).to(torch.bfloat16)
    up = torch.randn((count, n, rank), generator=g, device=DEV).to(torch.bfloat16)
    index = torch.randint(-1, count, (m,), generator=g, device=DEV).to(torch.int32)
    wp = nv.MXFP4Tensor(w.codes[:n], w.scales[:n])
    got = nv.mx_gemm_adapters(x[:m], wp, down, up, index)
    few = torch.cat([nv.mx_gemm_adapters(x[i:i + 1], wp, down, up, index[i:i + 1]) for i in range(m)])
    t = (x[:m].double().unsqueeze(1).abs() * down[index.long().clamp(min=0)].double().abs()).sum(2)
    bound = (t.unsqueeze(1) * up[index.long().clamp(min=0)].double().abs()).sum(2) + x[:m].double().abs() @ wd[0].abs().t()
    assert bool(((got - few).double().abs() <= 2 * (k / 8 + 3 * rank + 64) * 2.0 ** -24 * bound).all())
