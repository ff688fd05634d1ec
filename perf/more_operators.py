"""Products whose rows pick their weights, as timed workloads: the router that sorts rows by expert, the
products grouped by expert with ragged sizes, the expert layer for any number of tokens, and the low-rank
adapters of many requests beside a shared projection.  Weights are MXFP4, adapters bf16.

With ``own`` false, ``run`` computes each operator from elementary torch operations in float32; with
``own`` true it makes the package's calls.  ``exact`` gives the float64 result of the definition.

MXFP4: E2M1 codes (two per byte, even element in the low nibble) and one E8M0 byte b per 32
consecutive elements of a row; value = e2m1 * 2^(b - 127).
"""
import math

import torch

own = False

DEV = "cuda"
_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def _route(name, t, e, topk, src, renorm, masked):
    return {"name": name, "op": "route", "t": t, "e": e, "topk": topk, "src": src, "renorm": renorm, "masked": masked}


def _grouped(name, rows, groups, n, k, act, out, swiglu, gather):
    """n: rows of one group's weight; with swiglu half of them are gate rows and half up rows.  gather: rows of A that
    the products pick from (0: row i of A is row i of C)."""
    return {"name": name, "op": "grouped", "rows": rows, "groups": groups, "n": n, "k": k, "act": act, "out": out,
            "swiglu": swiglu, "gather": gather}


def _experts(name, t, e, topk, h, i, act, renorm, masked):
    return {"name": name, "op": "experts", "t": t, "e": e, "topk": topk, "h": h, "i": i, "act": act, "renorm": renorm,
            "masked": masked}


def _adapters(name, m, n, k, rank, count, act, out, requests):
    """requests: consecutive rows of one request share an adapter; 0: every row is a request."""
    return {"name": name, "op": "adapters", "m": m, "n": n, "k": k, "rank": rank, "count": count, "act": act, "out": out,
            "requests": requests}


def listed():
    return [
        # one decode token's router: launch latency
        _route("route_token", 1, 64, 8, "f32", True, False),
        # a mixed batch with a padded row and masked experts, bf16 scores full of ties
        _route("route_batch_masked", 515, 130, 3, "bf16", False, True),
        # the router of a long prompt
        _route("route_prompt", 16384, 128, 8, "bf16", True, False),
        # down product of a decode batch that is spread over many experts: a few rows each
        _grouped("grouped_w4a16_decode", 256, 64, 4096, 1536, "bf16", "f32", False, 0),
        # few experts, odd sizes, rows picked from a batch, activations quantized at call time
        _grouped("grouped_w4a4_odd", 777, 5, 1001, 2080, "mx", "f32", False, 389),
        # gate and up product of a prompt, weight-only
        _grouped("grouped_w4a16_swiglu", 4096, 16, 4096, 4096, "bf16", "bf16", True, 2048),
        # down product of a long prompt, activations quantized at call time
        _grouped("grouped_w4a4_prompt", 32768, 64, 4096, 2048, "mx", "bf16", False, 0),
        # the expert layer of a decode batch just past what the few-token layer takes
        _experts("experts_batch96", 96, 64, 8, 4096, 1536, "bf16", True, True),
        # the expert layer of a prompt, activations quantized
        _experts("experts_prompt", 4096, 64, 4, 4096, 1536, "mx", False, False),
        # one decode token with its adapter
        _adapters("adapters_token", 1, 4096, 4096, 16, 32, "bf16", "bf16", 0),
        # a decode batch, each row a request with an adapter of its own
        _adapters("adapters_batch48", 48, 12288, 4096, 16, 64, "bf16", "bf16", 0),
        # prompts of several requests packed into one call, activations quantized at call time
        _adapters("adapters_prompts", 4096, 4096, 4096, 64, 8, "mx", "bf16", 7),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "experts", "adapters", "adapters"])
    if op == "route":
        e = _logint(rng, 2, 512)
        c = _route("", _logint(rng, 1, 16384), e, rng.randint(1, min(16, e)), rng.choice(["f32", "bf16"]),
                   rng.random() < 0.5, rng.random() < 0.5)
        while c["t"] * (e + 16) > 16384 * 128:
            c["t"] //= 2
    elif op == "grouped":
        act, swiglu = rng.choice(["bf16", "mx"]), rng.random() < 0.5
        rows, groups = _logint(rng, 1, 32768), _logint(rng, 1, 128)
        n, k = (2 * _logint(rng, 1, 2048) if swiglu else _logint(rng, 1, 4096)), 32 * _logint(rng, 2, 128)
        while rows * n * k > 2 * 4096 * 4096 * 4096:
            rows = max(1, rows // 2)
        while groups * n * k > 64 * 4096 * 2048:
            groups = max(1, groups // 2)
        c = _grouped("", rows, groups, n, k, act, rng.choice(["f32", "bf16"]), swiglu,
                     rng.choice([0, max(1, rows // rng.randint(1, 8))]))
    elif op == "experts":
        e = _logint(rng, 2, 128)
        h, i = 32 * _logint(rng, 4, 128), 32 * _logint(rng, 2, 48)
        while e * h * i > 64 * 4096 * 1536:
            e //= 2
        t = _logint(rng, 1, 4096)
        while t * e * h * i > 4096 * 64 * 4096 * 1536:
            t //= 2
        c = _experts("", t, e, rng.randint(1, min(8, e)), h, i, rng.choice(["bf16", "mx"]), rng.random() < 0.5,
                     rng.random() < 0.5)
    else:
        m, n, k = _logint(rng, 1, 4096), _logint(rng, 1, 12288), 32 * _logint(rng, 2, 128)
        while m * n * k > 4096 * 4096 * 4096:
            m = max(1, m // 2)
        c = _adapters("", m, n, k, 8 * _logint(rng, 1, 16), _logint(rng, 1, 64), rng.choice(["bf16", "mx"]),
                      rng.choice(["f32", "bf16"]), rng.choice([0, _logint(rng, 1, 32)]))
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


def _through_mx(v):
    """float32 v as MXFP4 holds it."""
    v = v.contiguous()
    q, b = _mx_values(v)
    return (q * _pow2(b).unsqueeze(2)).view(v.shape)


def _expand32(codes, scales):
    """MXFP4 codes and scale bytes -> float32 values."""
    table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), dtype=torch.float32, device=codes.device)
    c = codes.to(torch.int32)
    v = torch.stack((table[c & 15], table[c >> 4]), dim=-1).view(codes.shape[0], -1, 32)
    return (v * _pow2(scales.to(torch.int32)).unsqueeze(2)).view(codes.shape[0], -1)


def _swiglu(g):
    i = g.shape[1] // 2
    return g[:, :i] * torch.sigmoid(g[:, :i]) * g[:, i:]


def _plain_topk(logits, topk, renorm):
    """ids [T, k] (-1 where fewer experts are left) and weights [T, k], taking the largest one at a time."""
    left = logits.to(torch.float32)
    top = left.amax(dim=1, keepdim=True)
    base = torch.where(top > float("-inf"), top, torch.zeros_like(top))
    p = torch.exp(left - base)
    ids, val = [], []
    idx = torch.arange(left.shape[1], device=left.device).view(1, -1)
    for _ in range(topk):
        m = left.amax(dim=1, keepdim=True)
        there = m > float("-inf")
        j = torch.where(left == m, idx, torch.full_like(idx, 1 << 30)).amin(dim=1, keepdim=True)
        ids.append(torch.where(there, j, torch.full_like(j, -1)))
        val.append(torch.where(there, torch.gather(p, 1, j), torch.zeros_like(m)))
        left = torch.where(idx == j, torch.full_like(left, float("-inf")), left)
    ids, val = torch.cat(ids, dim=1), torch.cat(val, dim=1)
    total = (val if renorm else p).sum(dim=1, keepdim=True)
    return ids, val / torch.where(total > 0, total, torch.ones_like(total))


def _plain_route(st):
    c = st["case"]
    ids, wts = _plain_topk(st["logits"], c["topk"], c["renorm"])
    flat = torch.where(ids < 0, torch.full_like(ids, c["e"]), ids).view(-1)
    hits = flat.view(1, -1) == torch.arange(c["e"], device=flat.device).view(-1, 1)  # [E, pairs]
    count = hits.sum(dim=1)
    ends = torch.cumsum(count, 0)
    offsets = torch.cat((torch.zeros_like(ends[:1]), ends))
    order = torch.cumsum(hits.to(torch.int32), dim=1)  # place within the expert, from one on
    n = flat.numel()
    at = torch.arange(n, device=flat.device)
    e = flat.clamp(max=c["e"] - 1)
    places = torch.where(flat < c["e"], offsets[e] + order[e, at] - 1, torch.full_like(flat, -1))
    rows = torch.full((n + 1,), -1, dtype=torch.int64, device=flat.device)
    rows.scatter_(0, torch.where(places >= 0, places, torch.full_like(places, n)), at // c["topk"])
    rows = torch.where(at < ends[-1], rows[:n], torch.full_like(at, -1))
    return (ids.to(torch.int32), wts, offsets.to(torch.int32), rows.to(torch.int32),
            places.view(ids.shape).to(torch.int32))


def _plain_grouped(st):
    c = st["case"]
    a = st["a"].to(torch.float32)
    if c["act"] == "mx":
        a = _through_mx(a)
    if st["rows"] is not None:
        a = a[st["rows"].to(torch.int64)]
    codes, scales = st["codes"].view(c["groups"], c["n"], -1), st["scales"].view(c["groups"], c["n"], -1)
    out = torch.empty((c["rows"], c["n"] // 2 if c["swiglu"] else c["n"]), dtype=st["dtype"], device=a.device)
    at = 0
    for g, size in enumerate(st["sizes"]):
        if size:
            v = torch.matmul(a[at:at + size], _expand32(codes[g], scales[g]).t())
            out[at:at + size] = (_swiglu(v) if c["swiglu"] else v).to(st["dtype"])
            at += size
    return out


def _plain_experts(st):
    """Every expert over every token; what an expert gives a token is rounded to bf16, weighted and summed in float32."""
    c = st["case"]
    e, h, i = c["e"], c["h"], c["i"]
    x = st["x"].to(torch.float32)
    if c["act"] == "mx":
        x = _through_mx(x)
    ids, wts = _plain_topk(st["logits"], c["topk"], c["renorm"])
    gu_c, gu_s = st["gu_codes"].view(e, 2 * i, -1), st["gu_scales"].view(e, 2 * i, -1)
    dn_c, dn_s = st["dn_codes"].view(e, h, -1), st["dn_scales"].view(e, h, -1)
    y = torch.zeros((c["t"], h), dtype=torch.float32, device=x.device)
    for j in range(e):
        a = _swiglu(x @ _expand32(gu_c[j], gu_s[j]).t())
        a = _through_mx(a) if c["act"] == "mx" else a.to(torch.bfloat16).to(torch.float32)
        z = (a @ _expand32(dn_c[j], dn_s[j]).t()).to(torch.bfloat16).to(torch.float32)
        y += torch.where(ids == j, wts, torch.zeros_like(wts)).sum(dim=1, keepdim=True) * z
    return y.to(torch.bfloat16)


def _plain_adapters(st):
    c = st["case"]
    x = st["a"].to(torch.float32)
    y = torch.matmul(_through_mx(x) if c["act"] == "mx" else x, _expand32(st["codes"], st["scales"]).t())
    idx = st["index"]
    if c["m"] * c["rank"] * (c["n"] + c["k"]) <= 1 << 26:  # few rows: each with its own adapter's matrices
        of = idx.clamp(min=0).to(torch.int64)
        t = (st["down"][of].to(torch.float32) * x.unsqueeze(1)).sum(dim=2) * st["scale"][of].unsqueeze(1)
        d = (st["up"][of].to(torch.float32) * t.unsqueeze(1)).sum(dim=2)
        return torch.where((idx >= 0).unsqueeze(1), y + d, y).to(st["dtype"])
    for j in range(c["count"]):
        t = torch.matmul(x, st["down"][j].to(torch.float32).t()) * st["scale"][j]
        d = torch.matmul(t, st["up"][j].to(torch.float32).t())
        y = torch.where((idx == j).unsqueeze(1), y + d, y)
    return y.to(st["dtype"])


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


def _scores(t, e, masked, g):
    """Router scores with some experts more popular than others; masked: a tenth of them at -inf, and a padded row."""
    logits = _randn((t, e), g) * 2 + _randn((1, e), g)
    if masked:
        logits[torch.rand((t, e), generator=g, device=DEV) < 0.1] = float("-inf")
        if t > 1:
            logits[t // 2] = float("-inf")
    return logits


def _tensor(codes, scales):
    import bit_gemm_nvfp4_amd as nv
    return nv.MXFP4Tensor(codes, scales)


def prepare(case, seed):
    g = _gen(seed)
    st = {"op": case["op"], "case": dict(case)}
    if case["op"] == "route":
        st["logits"] = _scores(case["t"], case["e"], case["masked"], g).to(_DTYPES[case["src"]])
        return st
    if case["op"] == "grouped":
        rows, groups = case["rows"], case["groups"]
        # ragged sizes: uneven shares, one group in eight without rows
        share = torch.rand(groups, generator=g, device=DEV) ** 2 + 0.05
        share[torch.rand(groups, generator=g, device=DEV) < 0.125] = 0
        share[int(torch.randint(groups, (1,), generator=g, device=DEV))] += 0.5
        pick = torch.multinomial(share, rows, replacement=True, generator=g)
        sizes = torch.bincount(pick, minlength=groups)
        st["sizes"] = sizes.tolist()
        st["offsets"] = torch.cat((torch.zeros_like(sizes[:1]), torch.cumsum(sizes, 0))).to(torch.int32)
        n_a = case["gather"] or rows
        st["a"] = _acts(n_a, case["k"], g)
        st["rows"] = (torch.randint(n_a, (rows,), generator=g, device=DEV).to(torch.int32) if case["gather"] else None)
        st["dtype"] = _DTYPES[case["out"]]
        st["codes"], st["scales"] = _weight(groups * case["n"], case["k"], g)
        if own:
            st["w"] = _tensor(st["codes"], st["scales"])
        return st
    if case["op"] == "experts":
        t, e, h, i = case["t"], case["e"], case["h"], case["i"]
        gu, dn = _weight(e * 2 * i, h, g), _weight(e * h, i, g)
        st.update(x=_acts(t, h, g), logits=_scores(t, e, case["masked"], g), gu_codes=gu[0], gu_scales=gu[1],
                  dn_codes=dn[0], dn_scales=dn[1])
        if own:
            st["w_gate_up"], st["w_down"] = _tensor(*gu), _tensor(*dn)
        return st
    m, n, k, r, count = case["m"], case["n"], case["k"], case["rank"], case["count"]
    st["codes"], st["scales"] = _weight(n, k, g)
    st["a"], st["dtype"] = _acts(m, k, g), _DTYPES[case["out"]]
    st["down"] = (_randn((count, r, k), g) / math.sqrt(k)).to(torch.bfloat16)
    st["up"] = (_randn((count, n, r), g) * 0.05).to(torch.bfloat16)
    st["scale"] = torch.rand(count, generator=g, device=DEV) + 0.5
    # one request in eight has no adapter (-1)
    requests = case["requests"] or m
    of = torch.randint(count, (requests,), generator=g, device=DEV)
    of = torch.where(torch.rand(requests, generator=g, device=DEV) < 0.125, torch.full_like(of, -1), of)
    if case["requests"]:  # ragged prompts one after the other
        cut = torch.sort(torch.randint(m + 1, (requests - 1,), generator=g, device=DEV))[0]
        of = of[torch.searchsorted(cut, torch.arange(m, device=DEV), right=True)]
    st["index"] = of.to(torch.int32)
    if own:
        st["w"] = _tensor(st["codes"], st["scales"])
    return st


def run(state):
    if not own:
        return {"route": _plain_route, "grouped": _plain_grouped, "experts": _plain_experts,
                "adapters": _plain_adapters}[state["op"]](state)
    import bit_gemm_nvfp4_amd as nv
    c = state["case"]
    if state["op"] == "route":
        r = nv.mx_route(state["logits"], c["topk"], renormalize=c["renorm"])
        return r.ids, r.weights, r.offsets, r.rows, r.places
    if state["op"] == "grouped":
        a = nv.mx_quantize(state["a"]) if c["act"] == "mx" else state["a"]
        return nv.mx_grouped_gemm(a, state["w"], state["offsets"], rows=state["rows"], swiglu=c["swiglu"],
                                  dtype=state["dtype"])
    if state["op"] == "experts":
        return nv.mx_experts(state["x"], state["logits"], state["w_gate_up"], state["w_down"], c["topk"],
                             renormalize=c["renorm"], quantize_acts=c["act"] == "mx", dtype=torch.bfloat16)
    a_q = nv.mx_quantize(state["a"]) if c["act"] == "mx" else None
    return nv.mx_gemm_adapters(state["a"], state["w"], state["down"], state["up"], state["index"], scales=state["scale"],
                               a_q=a_q, dtype=state["dtype"])


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without
# ------------------------------------------------------------------------------------------------
def _reached(of, tries):
    """Distinct ones of `of` that `tries` independent even choices reach."""
    return of * (1 - (1 - 1 / of) ** tries)


def work(case):
    bits = 17 / 32  # bytes per MXFP4 element: half a byte and its share of a scale byte
    if case["op"] == "route":
        t, e, k = case["t"], case["e"], case["topk"]
        return {"bytes": t * e * (4 if case["src"] == "f32" else 2) + 16 * t * k + 4 * (e + 1), "flops": t * e * 2}
    if case["op"] == "grouped":
        p, n, k = case["rows"], case["n"], case["k"]
        cols = n // 2 if case["swiglu"] else n
        picked = min(p, case["gather"] or p)
        return {"bytes": 2 * picked * k + bits * _reached(case["groups"], p) * n * k
                + (4 if case["out"] == "f32" else 2) * p * cols, "flops": 2 * p * n * k}
    if case["op"] == "experts":
        t, e, k, h, i = case["t"], case["e"], case["topk"], case["h"], case["i"]
        return {"bytes": _reached(e, t * k) * 3 * h * i * bits + t * (4 * h + 4 * e), "flops": 6 * t * k * h * i}
    m, n, k, r = case["m"], case["n"], case["k"], case["rank"]
    used = _reached(case["count"], case["requests"] or m)
    return {"bytes": 2 * m * k + bits * n * k + used * 2 * r * (n + k) + (4 if case["out"] == "f32" else 2) * m * n,
            "flops": 2 * m * n * k + 2 * m * r * (n + k)}


# ------------------------------------------------------------------------------------------------
# the definition in float64
# ------------------------------------------------------------------------------------------------
def _exp2_64(e):
    """2^e in float64 for whole e, from the exponent field."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _grid64(v):
    """float64 v -> MXFP4 values: the block exponent by frexp, the code by counting the midpoints
    passed (a tie passes the midpoint above an odd code only)."""
    blk = v.reshape(v.shape[0], -1, 32)
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


def _route64(logits, k, renorm):
    val, order = torch.sort(logits.double(), dim=1, descending=True, stable=True)
    base = val[:, :1]
    base = torch.where(base > float("-inf"), base, torch.zeros_like(base))
    ex = (val - base).exp()
    there = val[:, :k] > float("-inf")
    ids = torch.where(there, order[:, :k], torch.full_like(order[:, :k], -1))
    num = torch.where(there, ex[:, :k], torch.zeros_like(ex[:, :k]))
    den = (num if renorm else ex).sum(1, keepdim=True)
    return ids, num / torch.where(den > 0, den, torch.ones_like(den))


def _silu64(v):
    i = v.shape[1] // 2
    return v[:, :i] / (1 + torch.exp(-v[:, :i])) * v[:, i:]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        ids, wts = _route64(st["logits"], case["topk"], case["renorm"])
        flat, k = ids.flatten(), case["topk"]
        there = flat >= 0
        key = torch.where(there, flat, torch.full_like(flat, case["e"]))
        order = torch.sort(key, stable=True)[1]
        total = there.sum()
        rank = torch.empty_like(order)
        rank[order] = torch.arange(order.numel(), device=DEV)
        places = torch.where(there, rank, torch.full_like(rank, -1))
        rows = torch.where(torch.arange(order.numel(), device=DEV) < total, order // k, torch.full_like(order, -1))
        offsets = torch.searchsorted(key[order], torch.arange(case["e"] + 1, device=DEV))
        return (ids.int(), wts, offsets.int(), rows.int(), places.view(ids.shape).int())
    if case["op"] == "grouped":
        a = st["a"].double()
        if case["act"] == "mx":
            a = _grid64(a)
        outs, lo = [], 0
        for g in range(case["groups"]):
            hi = int(st["offsets"][g + 1])
            part = a[lo:hi] if st["rows"] is None else a.index_select(0, st["rows"][lo:hi].long())
            n = case["n"]
            v = part @ _decode64(st["codes"][g * n:(g + 1) * n], st["scales"][g * n:(g + 1) * n]).t()
            outs.append(_silu64(v) if case["swiglu"] else v)
            lo = hi
        return torch.cat(outs)
    if case["op"] == "experts":
        h, i = case["h"], case["i"]
        ids, wts = _route64(st["logits"], case["topk"], case["renorm"])
        x = st["x"].double()
        if case["act"] == "mx":
            x = _grid64(x)
        y = torch.zeros((case["t"], h), dtype=torch.float64, device=DEV)
        for j in torch.unique(ids[ids >= 0]).tolist():
            rows, slot = (ids == j).nonzero(as_tuple=True)
            gu = _decode64(st["gu_codes"][j * 2 * i:(j + 1) * 2 * i], st["gu_scales"][j * 2 * i:(j + 1) * 2 * i])
            a = _silu64(x[rows] @ gu.t())
            a = _grid64(a) if case["act"] == "mx" else a.bfloat16().double()
            z = a @ _decode64(st["dn_codes"][j * h:(j + 1) * h], st["dn_scales"][j * h:(j + 1) * h]).t()
            y[rows] += wts[rows, slot].unsqueeze(1) * z.bfloat16().double()
        return y
    x = st["a"].double()
    y = (_grid64(x) if case["act"] == "mx" else x) @ _decode64(st["codes"], st["scales"]).t()
    for j in range(case["count"]):
        rows = (st["index"] == j).nonzero().flatten()
        if rows.numel():
            t = x[rows] @ st["down"][j].double().t()
            y[rows] += float(st["scale"][j]) * (t @ st["up"][j].double().t())
    return y
