"""The MXFP4 operators as timed workloads: block quantization with a power-of-two scale per 32
elements, the product with MXFP4 weights, and the mixture-of-experts layer for a few tokens.

With ``own`` false, ``run`` computes each operator from elementary torch operations in float32; with
``own`` true it makes the package's calls.  ``exact`` gives the float64 result of the definition.

MXFP4: E2M1 codes (two per byte, even element in the low nibble) and one E8M0 byte b per 32
consecutive elements of a row; value = e2m1 * 2^(b - 127).
"""
import math

import torch

own = False

DEV = "cuda"
_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _quant(name, rows, cols, src, pad=0):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "src": src, "pad": pad}


def _gemm(name, m, n, k, act, out):
    return {"name": name, "op": "gemm", "m": m, "n": n, "k": k, "act": act, "out": out}


def _moe(name, t, e, topk, h, i, renorm, masked):
    return {"name": name, "op": "moe", "t": t, "e": e, "topk": topk, "h": h, "i": i, "renorm": renorm,
            "masked": masked}


def listed():
    return [
        # one decode token's activations: launch latency
        _quant("quantize_token", 1, 4096, "bf16"),
        # a ragged batch of activations that is a view into a wider buffer
        _quant("quantize_acts_strided", 517, 4096, "bf16", pad=64),
        # an MLP gate weight quantized from its fp32 master
        _quant("quantize_weight_f32", 12288, 4096, "f32"),
        # an MLP down weight requantized from FP8 with its tensor scale
        _quant("requantize_weight_fp8", 4096, 12288, "e4m3"),
        # one token through the gate projection, weight-only
        _gemm("gemm_w4a16_token", 1, 12288, 4096, "bf16", "bf16"),
        # a small decode batch through the down projection
        _gemm("gemm_w4a16_batch13", 13, 4096, 12288, "bf16", "f32"),
        # a prompt of 512 through the down projection, weight-only
        _gemm("gemm_w4a16_prompt", 512, 4096, 12288, "bf16", "bf16"),
        # a few rows, odd output width, activations quantized at call time
        _gemm("gemm_w4a4_rows5", 5, 4099, 4096, "mx", "f32"),
        # a prompt of 512 through the gate projection, activations quantized at call time
        _gemm("gemm_w4a4_prompt", 512, 12288, 4096, "mx", "f32"),
        # a long prompt (or a 1024 x 1024 image's latents): the largest product
        _gemm("gemm_w4a4_long", 4096, 12288, 4096, "mx", "bf16"),
        # one decode token through a layer of 64 experts
        _moe("moe_token", 1, 64, 8, 4096, 1536, True, False),
        # a decode batch with a padded row and masked experts, weights from the softmax over all experts
        _moe("moe_batch33", 33, 64, 4, 4096, 1536, False, True),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemm", "moe"])
    if op == "quantize":
        src = rng.choice(["f32", "bf16", "f16", "e4m3"])
        cols = 32 * _logint(rng, 1, 384)
        rows = _logint(rng, 1, min(18432, 12288 * 4096 // cols))
        c = _quant("", rows, cols, src, pad=rng.choice([0, 0, 16, 48]))
    elif op == "gemm":
        m, n, k = _logint(rng, 1, 4096), _logint(rng, 1, 12288), 32 * _logint(rng, 2, 384)
        while m * n * k > 4096 * 12288 * 4096:
            m = max(1, m // 2)
        c = _gemm("", m, n, k, rng.choice(["bf16", "mx"]), rng.choice(["f32", "bf16"]))
    else:
        e = _logint(rng, 2, 128)
        h, i = 32 * _logint(rng, 4, 128), 32 * _logint(rng, 2, 48)
        while e * h * i > 64 * 4096 * 1536:
            e //= 2
        c = _moe("", _logint(rng, 1, 64), e, rng.randint(1, min(8, e)), h, i, rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------------
# the plain form (float32)
# ------------------------------------------------------------------------------------------------
def _scale_bytes(v):
    """E8M0 byte of each block of 32: 2^(floor(log2 max|v|) - 2), from the exponent bits."""
    amax = v.view(v.shape[0], -1, 32).abs().amax(dim=2)
    return ((amax.view(torch.int32) >> 23) - 2).clamp_(min=0)


def _pow2(e):
    """2^(e - 127) in float32 for 0 <= e <= 254 (e = 0: the subnormal 2^-127)."""
    return torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _round_e2m1(y):
    """|y| to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6 (ties to the even code, 6 beyond), signed."""
    a = y.abs().clamp_(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, y)


def _mx_values(v):
    """(values on the E2M1 grid [rows, blocks, 32], scale bytes [rows, blocks]) of float32 v."""
    b = _scale_bytes(v)
    y = v.view(v.shape[0], -1, 32) * _pow2(254 - b).unsqueeze(2)
    return _round_e2m1(y), b


def _expand32(codes, scales):
    """MXFP4 codes and scale bytes -> float32 values."""
    table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=torch.float32, device=codes.device)
    c = codes.to(torch.int32)
    v = torch.stack((table[c & 15], table[c >> 4]), dim=-1).view(codes.shape[0], -1, 32)
    return (v * _pow2(scales.to(torch.int32)).unsqueeze(2)).view(codes.shape[0], -1)


def _widen32(st):
    x = st["x"]
    if st["src"] == "e4m3":
        return x.view(torch.float8_e4m3fn).to(torch.float32) * st["src_scale"]
    return x.to(torch.float32)


def _plain_quantize(st):
    v = _widen32(st).contiguous()
    q, b = _mx_values(v)
    return (q * _pow2(b).unsqueeze(2)).view(v.shape).to(torch.bfloat16)


def _plain_gemm(st):
    a = st["a"].to(torch.float32)
    if st["act"] == "mx":
        q, b = _mx_values(a)
        a = (q * _pow2(b).unsqueeze(2)).view(a.shape)
    return torch.matmul(a, _expand32(st["codes"], st["scales"]).t()).to(st["dtype"])


def _plain_routing(logits, topk, renorm):
    """ids [T, k] (int32, -1 where fewer experts are left) and weights [T, k] by counting ranks."""
    t, e = logits.shape
    lj, le = logits.unsqueeze(1), logits.unsqueeze(2)
    idx = torch.arange(e, device=logits.device)
    ahead = (lj > le) | ((lj == le) & (idx.view(1, 1, e) < idx.view(1, e, 1)))
    rank = ahead.sum(dim=2)
    valid = logits > float("-inf")
    slot = torch.where(valid & (rank < topk), rank, torch.full_like(rank, topk))
    ids = torch.full((t, topk + 1), -1, dtype=torch.int64, device=logits.device)
    ids.scatter_(1, slot, idx.expand(t, e))
    ids = ids[:, :topk]
    top = logits.amax(dim=1, keepdim=True)
    p = torch.where(valid, torch.exp(logits - torch.where(top > float("-inf"), top, torch.zeros_like(top))),
                    torch.zeros_like(logits))
    chosen = torch.where(ids >= 0, torch.gather(p, 1, ids.clamp(min=0)), torch.zeros_like(p[:, :1]))
    total = (chosen if renorm else p).sum(dim=1, keepdim=True)
    return ids, chosen / torch.where(total > 0, total, torch.ones_like(total))


def _plain_moe(st):
    c = st["case"]
    t, e, k, h, i = c["t"], c["e"], c["topk"], c["h"], c["i"]
    x = st["x"].to(torch.float32)
    ids, wts = _plain_routing(st["logits"], k, c["renorm"])
    gu_c, gu_s = st["gu_codes"].view(e, 2 * i, -1), st["gu_scales"].view(e, 2 * i, -1)
    dn_c, dn_s = st["dn_codes"].view(e, h, -1), st["dn_scales"].view(e, h, -1)
    y = torch.zeros((t, h), dtype=torch.float32, device=x.device)
    if t * k <= e:  # the chosen experts, one pair of token and expert at a time
        flat = ids.clamp(min=0)
        for p in range(t):
            for r in range(k):
                j = flat[p, r].view(1)
                g = _expand32(gu_c.index_select(0, j)[0], gu_s.index_select(0, j)[0]) @ x[p]
                a = g[:i] * torch.sigmoid(g[:i]) * g[i:]
                y[p] += wts[p, r] * (_expand32(dn_c.index_select(0, j)[0], dn_s.index_select(0, j)[0]) @ a)
    else:  # every expert over every token
        for j in range(e):
            g = x @ _expand32(gu_c[j], gu_s[j]).t()
            a = g[:, :i] * torch.sigmoid(g[:, :i]) * g[:, i:]
            w = torch.where(ids == j, wts, torch.zeros_like(wts)).sum(dim=1, keepdim=True)
            y += (a * w) @ _expand32(dn_c[j], dn_s[j]).t()
    return y.to(torch.bfloat16), ids.to(torch.int32), wts


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _weight(rows, cols, g):
    """A Gaussian weight in MXFP4, made a band of rows at a time."""
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=DEV)
    band = max(1, (1 << 26) // cols)
    code_of = torch.zeros(13, dtype=torch.int32, device=DEV)  # twice the magnitude -> code
    for c, m in enumerate(_E2M1):
        code_of[int(2 * m)] = c
    for r in range(0, rows, band):
        q, b = _mx_values(_randn((min(band, rows - r), cols), g) * 0.02)
        n = code_of[(q.abs() * 2).to(torch.int32)] | (torch.signbit(q).to(torch.int32) << 3)
        n = n.view(n.shape[0], -1, 2)
        codes[r:r + band] = (n[:, :, 0] | (n[:, :, 1] << 4)).to(torch.uint8)
        scales[r:r + band] = b.to(torch.uint8)
    return codes, scales


def _acts(rows, cols, g):
    """Gaussian activations with one channel in a thousand twenty times larger."""
    a = _randn((rows, cols), g)
    hot = torch.rand(cols, generator=g, device=DEV) < 1e-3
    return torch.where(hot, a * 20, a).to(torch.bfloat16)


def _tensor(codes, scales):
    import bit_gemm_nvfp4_amd as nv
    return nv.MXFP4Tensor(codes, scales)


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quantize":
        rows, cols, pad, src = case["rows"], case["cols"], case["pad"], case["src"]
        st = {"op": "quantize", "src": src, "src_scale": None}
        v = _randn((rows, cols + pad), g)
        if src == "e4m3":
            w = v * 0.02
            s = (w.abs().amax() / 448).view(1)
            st["x"], st["src_scale"] = (w / s).to(torch.float8_e4m3fn).view(torch.uint8)[:, :cols], s
        else:
            if src == "f32":
                v = v * 0.02
            if rows > 64:
                v[rows // 2] = 0  # a pruned row, or a padded token
            st["x"] = v.to(_DTYPES[src])[:, :cols]
        return st
    if case["op"] == "gemm":
        codes, scales = _weight(case["n"], case["k"], g)
        st = {"op": "gemm", "act": case["act"], "a": _acts(case["m"], case["k"], g), "codes": codes, "scales": scales,
              "dtype": _DTYPES[case["out"]]}
        if own:
            st["w"] = _tensor(codes, scales)
        return st
    t, e, h, i = case["t"], case["e"], case["h"], case["i"]
    gu, dn = _weight(e * 2 * i, h, g), _weight(e * h, i, g)
    logits = _randn((t, e), g) * 2
    if case["masked"]:
        logits[torch.rand((t, e), generator=g, device=DEV) < 0.1] = float("-inf")
        if t > 1:
            logits[t // 2] = float("-inf")  # a padded row
    st = {"op": "moe", "case": dict(case), "x": _acts(t, h, g), "logits": logits, "gu_codes": gu[0], "gu_scales": gu[1],
          "dn_codes": dn[0], "dn_scales": dn[1]}
    if own:
        st["w_gate_up"], st["w_down"] = _tensor(*gu), _tensor(*dn)
    return st


def run(state):
    if not own:
        return {"quantize": _plain_quantize, "gemm": _plain_gemm, "moe": _plain_moe}[state["op"]](state)
    import bit_gemm_nvfp4_amd as nv
    if state["op"] == "quantize":
        return nv.mx_dequantize(nv.mx_quantize(state["x"], src_scale=state["src_scale"]), torch.bfloat16)
    if state["op"] == "gemm":
        a = nv.mx_quantize(state["a"]) if state["act"] == "mx" else state["a"]
        return nv.mx_gemm(a, state["w"], dtype=state["dtype"])
    c = state["case"]
    return nv.mx_moe(state["x"], state["logits"], state["w_gate_up"], state["w_down"], c["topk"],
                     renormalize=c["renorm"], dtype=torch.bfloat16, routing=True)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def work(case):
    bits = 17 / 32  # bytes per MXFP4 element: half a byte and its share of a scale byte
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        # read the source, write the codes and the values they stand for
        return {"bytes": n * ({"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}[case["src"]] + bits + 2), "flops": n * 2}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + bits * n * k + (4 if case["out"] == "f32" else 2) * m * n, "flops": 2 * m * n * k}
    t, e, k, h, i = case["t"], case["e"], case["topk"], case["h"], case["i"]
    experts = e * (1 - (1 - k / e) ** t)  # distinct experts that independent choices reach
    return {"bytes": experts * 3 * h * i * bits + t * (4 * h + 4 * e + 8 * k), "flops": 6 * t * k * h * i}


# ------------------------------------------------------------------------------------------------
# the definition in float64
# ------------------------------------------------------------------------------------------------
def _exp2_64(e):
    """2^e in float64 for whole e, from the exponent field."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _grid64(v):
    """float64 v -> MXFP4 values: the block exponent by frexp, the code by counting the midpoints
    passed (a tie passes the midpoint above an odd code only)."""
    blk = v.view(v.shape[0], -1, 32)
    amax = blk.abs().amax(dim=2, keepdim=True)
    ex = (torch.frexp(amax)[1] - 3).clamp(min=-127)
    ex = torch.where(amax > 0, ex, torch.full_like(ex, -127))
    scale = _exp2_64(ex)
    a = blk.abs() / scale
    mag = torch.zeros_like(a)
    for c in range(7):
        mid = (_E2M1[c] + _E2M1[c + 1]) / 2
        mag += ((a >= mid) if c % 2 else (a > mid)).to(torch.float64) * (_E2M1[c + 1] - _E2M1[c])
    return (torch.where(blk < 0, -mag, mag) * scale).view(v.shape)


def _decode64(codes, scales):
    lo, hi = (codes & 15).long(), (codes >> 4).long()
    nib = torch.stack((lo, hi), dim=2).view(codes.shape[0], -1)
    mag = torch.tensor(_E2M1, dtype=torch.float64, device=codes.device)[nib & 7]
    mag = torch.where(nib >= 8, -mag, mag)
    s = _exp2_64(scales.to(torch.int64) - 127)
    return mag * s.repeat_interleave(32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "quantize":
        if case["src"] == "e4m3":  # the source is widened with one float32 rounding by definition
            v = (st["x"].view(torch.float8_e4m3fn).double() * st["src_scale"].double()).float().double()
        else:
            v = st["x"].double()
        return _grid64(v.contiguous())
    if case["op"] == "gemm":
        a = st["a"].double()
        if case["act"] == "mx":
            a = _grid64(a)
        return a @ _decode64(st["codes"], st["scales"]).t()
    e, k, h, i = case["e"], case["topk"], case["h"], case["i"]
    x, logits = st["x"].double(), st["logits"].double()
    val, order = torch.sort(logits, dim=1, descending=True, stable=True)
    val, order = val[:, :k], order[:, :k]
    there = val > float("-inf")
    ids = torch.where(there, order, torch.full_like(order, -1))
    base = logits.amax(dim=1, keepdim=True)
    base = torch.where(base > float("-inf"), base, torch.zeros_like(base))
    num = torch.where(there, (val - base).exp(), torch.zeros_like(val))
    den = num.sum(1, keepdim=True) if case["renorm"] else (logits - base).exp().sum(1, keepdim=True)
    wts = num / torch.where(den > 0, den, torch.ones_like(den))
    y = torch.zeros((case["t"], h), dtype=torch.float64, device=x.device)
    for j in torch.unique(ids[ids >= 0]).tolist():
        rows = (ids == j).any(dim=1).nonzero().flatten()
        gu = _decode64(st["gu_codes"][j * 2 * i:(j + 1) * 2 * i], st["gu_scales"][j * 2 * i:(j + 1) * 2 * i])
        g = x[rows] @ gu.t()
        act = g[:, :i] / (1 + torch.exp(-g[:, :i])) * g[:, i:]
        dn = _decode64(st["dn_codes"][j * h:(j + 1) * h], st["dn_scales"][j * h:(j + 1) * h])
        w = torch.where(ids[rows] == j, wts[rows], torch.zeros_like(wts[rows])).sum(1, keepdim=True)
        y[rows] += w * (act @ dn.t())
    return y, ids.to(torch.int32), wts
