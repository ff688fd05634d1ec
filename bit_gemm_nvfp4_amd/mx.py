"""MXFP4 (E2M1 codes, one power-of-two E8M0 scale per 32 elements of a row): quantization, expansion,
the product with MXFP4 weights, the mixture-of-experts layer for a few tokens, and products whose rows pick
their weights: router, products grouped by expert, the layer for any number of tokens, adapters per request.

A thin ctypes binding over the entry points of ``include/mxfp4.h``; the package re-exports its names.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

from . import (_DT, _I32, _I64, _P, _SIGNATURES, _RESTYPES, _SZ, _check, _rows, _workspace, check_flags,
               load_library)

MX_OP_GEMM_BF16, MX_OP_GEMM_MX, MX_OP_MOE, MX_OP_ROUTE, MX_OP_GROUP_ROWS = 0, 1, 2, 3, 4
MX_BLOCK = 32
SKINNY_MAX_M = 16  # products of up to this many rows take no workspace
MOE_MAX_TOKENS, MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 64, 512, 16
GROUP_MAX_ROWS, MAX_GROUPS = 1 << 24, MOE_MAX_EXPERTS
ROUTE_ONE_LAUNCH = 16  # a router of up to this many rows takes no workspace
MX_EXPORTED = ["mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_moe", "mxfp4_workspace_size", "mxfp4_route",
               "mxfp4_group_rows", "mxfp4_grouped_gemm", "mxfp4_combine", "mxfp4_experts",
               "mxfp4_experts_workspace_size", "mxfp4_gemm_adapters", "mxfp4_adapters_workspace_size"]


class CMXTensor(ctypes.Structure):
    """Mirror of `mxfp4_tensor`."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


_PX = ctypes.POINTER(CMXTensor)
_SIGNATURES.update({
    "mxfp4_quantize": [_P, _I32, _I64, _P, _PX, _P, _P],
    "mxfp4_dequantize": [_PX, _P, _I32, _I64, _P],
    "mxfp4_gemm": [_P, _PX, _I64, _I64, _PX, _P, _I32, _I64, _P, _SZ, _P],
    "mxfp4_moe": [_P, _I64, _I64, _P, _I32, _I64, _I64, _I32, _I32, _PX, _PX, _P, _I32, _I64, _P, _P, _P, _SZ, _P],
    "mxfp4_workspace_size": [_I32, _I64, _I64, _I64],
    "mxfp4_route": [_P, _I32, _I64, _I64, _I64, _I32, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P],
    "mxfp4_group_rows": [_P, _I64, _I32, _I64, _P, _P, _P, _P, _SZ, _P],
    "mxfp4_grouped_gemm": [_P, _PX, _I64, _I64, _P, _P, _I64, _I64, _PX, _I32, _P, _I32, _I64, _PX, _P],
    "mxfp4_combine": [_P, _I32, _I64, _I64, _P, _P, _I64, _I32, _I64, _P, _I32, _I64, _P],
    "mxfp4_experts": [_P, _I64, _I64, _P, _I32, _I64, _I64, _I32, _I32, _I32, _PX, _PX, _P, _I32, _I64, _P, _P, _P, _SZ,
                      _P],
    "mxfp4_experts_workspace_size": [_I64, _I64, _I32, _I64, _I64, _I32, _I32],
    "mxfp4_gemm_adapters": [_P, _PX, _I64, _I64, _PX, _P, _I64, _I64, _P, _P, _P, _P, _I32, _I64, _P, _SZ, _P],
    "mxfp4_adapters_workspace_size": [_I64, _I64, _I64, _I64, _I64, _I32],
})
for _name in ("mxfp4_workspace_size", "mxfp4_experts_workspace_size", "mxfp4_adapters_workspace_size"):
    _RESTYPES[_name] = _SZ


@dataclass
class MXFP4Tensor:
    """Packed MXFP4 tensor of logical shape [rows, cols], cols a multiple of 32: codes [rows, cols/2]
    uint8 (element 2j in the low nibble of byte j) and scales [rows, cols/32] uint8 (E8M0: the scale is
    2^(byte - 127), 255 marks a block with a non-finite source).  `flags` is the device int32 word
    given to the producing quantize call (bit 0: non-finite input), or None."""
    codes: torch.Tensor
    scales: torch.Tensor
    flags: torch.Tensor | None = None

    @property
    def shape(self):
        return (self.codes.shape[0], self.codes.shape[1] * 2)

    @staticmethod
    def empty(rows: int, cols: int, device) -> "MXFP4Tensor":
        assert cols % MX_BLOCK == 0, f"MXFP4 needs a multiple of {MX_BLOCK} columns, not {cols}"
        return MXFP4Tensor(torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
                           torch.empty((rows, cols // MX_BLOCK), dtype=torch.uint8, device=device))

    def c(self) -> CMXTensor:
        codes, scales = self.codes, self.scales
        r, half = codes.shape
        assert half % (MX_BLOCK // 2) == 0 and scales.shape == (r, half // (MX_BLOCK // 2)), \
            f"MXFP4 scales: shape {tuple(scales.shape)}, expected {(r, half / (MX_BLOCK // 2))}"
        assert codes.is_cuda and codes.dtype is torch.uint8 and scales.dtype is torch.uint8 and \
            scales.device == codes.device, "MXFP4 codes and scales must be uint8 device tensors on one device"
        assert codes.is_contiguous() and scales.is_contiguous(), "MXFP4 codes and scales must be dense"
        return CMXTensor(codes.data_ptr(), scales.data_ptr(), r, half * 2)


# The binding's own time is most of a small call's, so it takes the raw current stream of the device and
# switches devices only when the tensors are not on the current one.  Like the library, what torch has only in
# builds for GPUs is looked up at the first call.
_raw_stream = None
_current_device = torch.cuda.current_device


_functions: dict = {}


def _function(name: str):
    global _raw_stream
    _raw_stream = torch._C._cuda_getCurrentRawStream
    fn = _functions[name] = getattr(load_library(), name)
    return fn


def _call(name: str, device: torch.device, *args) -> None:
    """Call entry point `name` with `args` and the current stream of `device`.  The library launches on
    the current device, so `device` is made current for the call if it is not."""
    fn = _functions.get(name) or _function(name)
    index = device.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        _check(status, name)


def _opt(t: torch.Tensor | None, device: torch.device, name: str, dtype: torch.dtype | None = None):
    """Address of an optional tensor argument on `device`; of a single `dtype` when one is given."""
    if t is None:
        return None
    assert t.device == device and (dtype is None or t.dtype is dtype and t.numel() == 1), \
        f"{name}: {t.numel()} x {t.dtype} on {t.device}"
    return t.data_ptr()


def _nbytes(t: torch.Tensor | None) -> int:
    if t is None:
        return 0
    assert t.is_contiguous(), "workspace: a dense tensor is required"
    return t.numel() * t.element_size()


def _out(out: torch.Tensor | None, rows: int, cols: int, dtype: torch.dtype, device, what: str):
    """The output matrix (allocated when not given), its row stride and the C dtype."""
    if out is None:
        assert dtype is torch.float32 or dtype is torch.bfloat16, f"{what}: dtype {dtype} not offered"
        return torch.empty((rows, cols), dtype=dtype, device=device), cols, _DT[dtype]
    assert out.device == device and out.dtype in (torch.float32, torch.bfloat16) and out.shape[0] == rows, \
        f"{what}: {tuple(out.shape)} {out.dtype} on {out.device}"
    return out, _rows(out, what, cols), _DT[out.dtype]


def mx_workspace_size(op: int, m: int, n: int, k: int) -> int:
    return int(load_library().mxfp4_workspace_size(op, m, n, k))


def mx_quantize(x: torch.Tensor, src_scale: torch.Tensor | None = None, flags: torch.Tensor | None = None,
                out: MXFP4Tensor | None = None, check: bool = False) -> MXFP4Tensor:
    """Quantize a 2-D device tensor (fp32, bf16, fp16, or float8_e4m3fn / uint8 E4M3 bytes; columns a
    multiple of 32) to MXFP4 in one pass: per 32-element block the scale 2^(floor(log2 max|x|) - 2), codes
    rounded to nearest even, saturating at 6.  A block with a NaN or infinity reads back as NaN.
    src_scale: device fp32 [1] per-tensor scale of an E4M3 source.  flags: device int32 [1] that the
    call ORs bit 0 into on non-finite input.  check: synchronise and raise on non-finite input."""
    ld = _rows(x, "x")
    rows, cols = x.shape
    dev = x.device
    if out is None:
        out = MXFP4Tensor.empty(rows, cols, dev)
        ct = CMXTensor(out.codes.data_ptr(), out.scales.data_ptr(), rows, cols)
    elif out.shape != (rows, cols) or out.codes.device != dev:
        raise AssertionError(f"out: shape {out.shape} on {out.codes.device}, expected {(rows, cols)} on {dev}")
    else:
        ct = out.c()
    if flags is None and check:
        flags = torch.zeros(1, dtype=torch.int32, device=dev)
    _call("mxfp4_quantize", dev, x.data_ptr(), _DT[x.dtype], ld, _opt(src_scale, dev, "src_scale", torch.float32),
          ctypes.byref(ct), _opt(flags, dev, "flags", torch.int32))
    out.flags = flags
    if check:
        check_flags(flags, "mxfp4_quantize")
    return out


def mx_dequantize(q: MXFP4Tensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Expand MXFP4 to bf16 or fp32 (exact)."""
    rows, cols = q.shape
    dev = q.codes.device
    out, ld, dt = _out(out, rows, cols, dtype, dev, "out")
    _call("mxfp4_dequantize", dev, ctypes.byref(q.c()), out.data_ptr(), dt, ld)
    return out


def _gemm_workspace(op: int, m: int, n: int, k: int, device: torch.device) -> torch.Tensor | None:
    if device.index == torch.cuda.current_device():  # the size is planned for the current device
        return _workspace(mx_workspace_size(op, m, n, k), device)
    with torch.cuda.device(device.index):
        return _workspace(mx_workspace_size(op, m, n, k), device)


def mx_gemm_workspace(a: torch.Tensor | MXFP4Tensor, w: MXFP4Tensor) -> torch.Tensor | None:
    """A workspace for mx_gemm(a, w), for callers that keep one (None when the product needs none).  Its
    contents do not matter; calls that share one must be ordered (same stream, or events)."""
    op = MX_OP_GEMM_MX if isinstance(a, MXFP4Tensor) else MX_OP_GEMM_BF16
    return _gemm_workspace(op, a.shape[0], w.shape[0], w.shape[1], w.codes.device)


def mx_gemm(a: torch.Tensor | MXFP4Tensor, w: MXFP4Tensor, dtype: torch.dtype = torch.float32,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C [M, N] (fp32 or bf16) = A . W^T with MXFP4 weights [N, K].  `a` is an MXFP4Tensor [M, K] (W4A4: FP4
    matrix instructions) or a bf16 tensor [M, K] (W4A16).  fp32 sums, rounded once."""
    assert isinstance(w, MXFP4Tensor), "w: an MXFP4Tensor is required"
    n, k = w.shape
    dev = w.codes.device
    m = a.shape[0]
    if isinstance(a, MXFP4Tensor):
        assert a.shape[1] == k and a.codes.device == dev, f"a: {a.shape} on {a.codes.device}, expected {k} columns on {dev}"
        a_ct, a_ptr, lda, op = ctypes.byref(a.c()), None, k, MX_OP_GEMM_MX
    else:
        assert isinstance(a, torch.Tensor) and a.dtype is torch.bfloat16 and a.device == dev, \
            f"a: a bf16 tensor or an MXFP4Tensor on {dev} is required"
        lda = _rows(a, "a", k)
        a_ct, a_ptr, op = None, a.data_ptr(), MX_OP_GEMM_BF16
    out, ldc, dt = _out(out, m, n, dtype, dev, "out")
    if workspace is None and m > SKINNY_MAX_M:  # none needed below
        workspace = _gemm_workspace(op, m, n, k, dev)
    _call("mxfp4_gemm", dev, a_ptr, a_ct, m, lda, ctypes.byref(w.c()), out.data_ptr(), dt, ldc,
          _opt(workspace, dev, "workspace"), _nbytes(workspace))
    return out


def mx_moe_workspace(tokens: int, top_k: int, w_gate_up: MXFP4Tensor, w_down: MXFP4Tensor) -> torch.Tensor | None:
    """A workspace for mx_moe (None without tokens).  Its contents do not matter; calls that share one
    must be ordered (same stream, or events)."""
    nbytes = mx_workspace_size(MX_OP_MOE, tokens * top_k, w_gate_up.shape[1], w_down.shape[1])
    return _workspace(nbytes, w_down.codes.device)


def mx_moe(x: torch.Tensor, logits: torch.Tensor, w_gate_up: MXFP4Tensor, w_down: MXFP4Tensor, top_k: int,
           renormalize: bool = True, dtype: torch.dtype = torch.bfloat16, routing: bool = False,
           out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Mixture-of-experts layer for up to 64 tokens: y[t] = sum_e p[t, e] Wd[e] (silu(Wg[e] x[t]) * (Wu[e]
    x[t])) over the top_k largest of logits[t] (ties to the lowest expert).

    x [T, H] bf16; logits [T, E] fp32 or bf16 (-inf masks an expert; a row that is all -inf gives 0; one
    with NaN or +inf gives NaN); w_gate_up [E * 2I, H] (per expert I gate rows, then I up rows) and
    w_down [E * H, I], experts stacked.  p is the softmax over the chosen logits (renormalize), or the
    chosen entries of the softmax over all of them.  Returns y [T, H], or with routing=True (y, ids,
    weights): ids [T, top_k] int32 in descending order of logit and their p, -1 and 0 where a row has fewer."""
    dev = x.device
    assert x.dtype is torch.bfloat16, f"x: bf16, not {x.dtype}"
    assert logits.dtype in (torch.float32, torch.bfloat16), f"logits: fp32 or bf16, not {logits.dtype}"
    ld_x, ld_l = _rows(x, "x", w_gate_up.shape[1]), _rows(logits, "logits")
    t, h = x.shape
    assert logits.shape[0] == t, f"logits: {logits.shape[0]} rows, expected {t}"
    assert logits.device == dev and w_gate_up.codes.device == dev and w_down.codes.device == dev, "one device per call"
    out, ld_y, dt = _out(out, t, h, dtype, dev, "out")
    ids = weights = None
    if routing:
        ids = torch.empty((t, top_k), dtype=torch.int32, device=dev)
        weights = torch.empty((t, top_k), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = mx_moe_workspace(t, top_k, w_gate_up, w_down)
    _call("mxfp4_moe", dev, x.data_ptr(), t, ld_x, logits.data_ptr(), _DT[logits.dtype], ld_l, logits.shape[1], top_k,
          1 if renormalize else 0, ctypes.byref(w_gate_up.c()), ctypes.byref(w_down.c()), out.data_ptr(), dt, ld_y,
          _opt(ids, dev, "ids"), _opt(weights, dev, "weights"), _opt(workspace, dev, "workspace"), _nbytes(workspace))
    return (out, ids, weights) if routing else out


# ------------------------------------------------------------------------------------------------
# products whose rows pick their weights
# ------------------------------------------------------------------------------------------------
@dataclass
class Grouping:
    """Rows sorted by group (an expert): group g has the positions offsets[g] .. offsets[g + 1] - 1 (int32 [groups + 1]);
    rows [tokens * per_token] int32 is the token at each position, -1 behind the last group's; places [tokens,
    per_token] int32 the position of each choice, -1 where there is none.  From mx_route also the choices: ids [tokens,
    top_k] int32 and their weights fp32."""
    offsets: torch.Tensor
    rows: torch.Tensor
    places: torch.Tensor | None = None
    ids: torch.Tensor | None = None
    weights: torch.Tensor | None = None


def _words(t: torch.Tensor, what: str, device: torch.device, dtype: torch.dtype, *shape) -> int:
    """Address of a dense tensor argument of the given type and shape."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise AssertionError(f"{what}: a dense {dtype} tensor {shape} on {device} is required, not {tuple(t.shape)} {t.dtype} on {t.device}")


def mx_route(logits: torch.Tensor, top_k: int, renormalize: bool = True,
             workspace: torch.Tensor | None = None) -> Grouping:
    """The router of a mixture-of-experts layer: the top_k largest of each row of logits [T, E] (fp32 or bf16; ties to
    the lowest expert, -inf masks an expert), their softmax weights (over the chosen logits, or with renormalize=False
    over all of the row's), and the tokens sorted by expert, in their order within an expert.  A row with a NaN or +inf
    chooses no expert and has NaN weights."""
    dev = logits.device
    assert logits.dtype in (torch.float32, torch.bfloat16), f"logits: fp32 or bf16, not {logits.dtype}"
    ld = _rows(logits, "logits")
    t, e = logits.shape
    assert top_k >= 1, f"top_k: at least 1, not {top_k}"
    n = t * top_k
    # (one allocation, divided)
    ids, places, rows, offsets = torch.empty(3 * n + e + 1, dtype=torch.int32, device=dev).split((n, n, n, e + 1))
    ids, places = ids.view(t, top_k), places.view(t, top_k)
    weights = torch.empty((t, top_k), dtype=torch.float32, device=dev)
    if workspace is None and t > ROUTE_ONE_LAUNCH:  # none needed below
        workspace = _workspace(mx_workspace_size(MX_OP_ROUTE, t, top_k, e), dev)
    _call("mxfp4_route", dev, logits.data_ptr(), _DT[logits.dtype], t, ld, e, top_k, 1 if renormalize else 0, ids.data_ptr(),
          weights.data_ptr(), offsets.data_ptr(), rows.data_ptr(), places.data_ptr(), _opt(workspace, dev, "workspace"),
          _nbytes(workspace))
    return Grouping(offsets, rows, places, ids, weights)


def mx_group_rows(ids: torch.Tensor, groups: int, workspace: torch.Tensor | None = None) -> Grouping:
    """Sort tokens by the groups that they name: ids int32 [T, per_token] (or [T]) in 0 .. groups - 1, any other value
    being no choice.  A token may name a group more than once."""
    assert ids.is_cuda and ids.dtype is torch.int32 and ids.dim() in (1, 2) and ids.is_contiguous(), \
        "ids: a dense int32 device tensor [tokens] or [tokens, per_token] is required"
    t, per = ids.shape[0], 1 if ids.dim() == 1 else ids.shape[1]
    dev = ids.device
    offsets = torch.empty(max(groups, 0) + 1, dtype=torch.int32, device=dev)
    rows = torch.empty(t * per, dtype=torch.int32, device=dev)
    places = torch.empty((t, per), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = _workspace(mx_workspace_size(MX_OP_GROUP_ROWS, t, per, groups), dev)
    _call("mxfp4_group_rows", dev, ids.data_ptr(), t, per, groups, offsets.data_ptr(), rows.data_ptr(), places.data_ptr(),
          _opt(workspace, dev, "workspace"), _nbytes(workspace))
    return Grouping(offsets, rows, places)


def mx_grouped_gemm(a: torch.Tensor | MXFP4Tensor, w: MXFP4Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                    swiglu: bool = False, dtype: torch.dtype = torch.float32,
                    out: torch.Tensor | MXFP4Tensor | None = None) -> torch.Tensor | MXFP4Tensor:
    """Products grouped by expert, of any sizes: for offsets[g] <= i < offsets[g + 1] (int32 [groups + 1], on the
    device), C[i] = A[rows[i]] . W[g]^T, or with swiglu silu(A[rows[i]] . Wg[g]^T) * (A[rows[i]] . Wu[g]^T).

    a: MXFP4Tensor (W4A4) or bf16 [R, K] (W4A16); rows: int32, the row of A of each row of C (all of A's, in order,
    without it; one outside A counts as zeros); w [groups * N, K], groups stacked (swiglu: N / 2 gate rows, then N / 2 up
    rows, per group).  Returns C [len(rows) or R, N or N / 2], fp32 or bf16; with swiglu `out` may be an MXFP4Tensor, which
    is quantized from the fp32 values.  Rows outside every group (those behind the last one, where
    a router has masked experts) are left as they are in `out`; without `out` they hold anything, NaN included."""
    assert isinstance(w, MXFP4Tensor), "w: an MXFP4Tensor is required"
    wr, k = w.shape
    dev = w.codes.device
    assert offsets.dim() == 1 and offsets.numel() >= 2, f"offsets: [groups + 1] is required, not {tuple(offsets.shape)}"
    groups = offsets.numel() - 1
    parts = groups * (2 if swiglu else 1)
    assert wr % parts == 0, f"w: {wr} rows do not make {groups} groups"
    n = wr // parts
    if isinstance(a, MXFP4Tensor):
        assert a.shape[1] == k and a.codes.device == dev, f"a: {a.shape} on {a.codes.device}, expected {k} columns on {dev}"
        a_ct, a_ptr, lda = ctypes.byref(a.c()), None, k
    else:
        assert isinstance(a, torch.Tensor) and a.dtype is torch.bfloat16 and a.device == dev, \
            f"a: a bf16 tensor or an MXFP4Tensor on {dev} is required"
        lda = _rows(a, "a", k)
        a_ct, a_ptr = None, a.data_ptr()
    m = a.shape[0] if rows is None else rows.numel()
    map_ptr = None if rows is None else _words(rows, "rows", dev, torch.int32, m)
    off_ptr = _words(offsets, "offsets", dev, torch.int32, groups + 1)
    if isinstance(out, MXFP4Tensor):
        assert swiglu and out.shape == (m, n) and out.codes.device == dev, \
            f"out: MXFP4 {out.shape} on {out.codes.device}, expected {(m, n)} on {dev}, with swiglu"
        c_ct, c_ptr, ldc, dt = ctypes.byref(out.c()), None, n, 0
    else:
        out, ldc, dt = _out(out, m, n, dtype, dev, "out")
        c_ct, c_ptr = None, out.data_ptr()
    _call("mxfp4_grouped_gemm", dev, a_ptr, a_ct, a.shape[0], lda, map_ptr, off_ptr, groups, m, ctypes.byref(w.c()),
          1 if swiglu else 0, c_ptr, dt, ldc, c_ct)
    if c_ct is not None:
        out.flags = None  # a word of an earlier mx_quantize does not speak for these values
    return out


def mx_combine(z: torch.Tensor, places: torch.Tensor, weights: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
               out: torch.Tensor | None = None) -> torch.Tensor:
    """y[t] = sum_j weights[t, j] z[places[t, j]] (fp32 sums in the order of j): what a token's choices gave back.  z [P, N]
    fp32 or bf16; places int32 and weights fp32 [T, top_k]; a place outside z counts as a row of zeros."""
    assert z.dtype in (torch.float32, torch.bfloat16), f"z: fp32 or bf16, not {z.dtype}"
    dev = z.device
    ld = _rows(z, "z")
    assert places.dim() == 2, f"places: [tokens, top_k] is required, not {tuple(places.shape)}"
    t, k = places.shape
    cols = z.shape[1]
    out, ld_y, dt = _out(out, t, cols, dtype, dev, "out")
    _call("mxfp4_combine", dev, z.data_ptr(), _DT[z.dtype], z.shape[0], ld, _words(places, "places", dev, torch.int32, t, k),
          _words(weights, "weights", dev, torch.float32, t, k), t, k, cols, out.data_ptr(), dt, ld_y)
    return out


def mx_experts_workspace(tokens: int, experts: int, top_k: int, w_gate_up: MXFP4Tensor, w_down: MXFP4Tensor,
                         quantize_acts: bool = True, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor | None:
    """A workspace for mx_experts (None without tokens).  Its contents do not matter; calls that share one must be ordered
    (same stream, or events)."""
    nbytes = int(load_library().mxfp4_experts_workspace_size(tokens, experts, top_k, w_gate_up.shape[1], w_down.shape[1],
                                                             1 if quantize_acts else 0, _DT[dtype]))
    return _workspace(nbytes, w_down.codes.device)


def mx_experts(x: torch.Tensor, logits: torch.Tensor, w_gate_up: MXFP4Tensor, w_down: MXFP4Tensor, top_k: int,
               renormalize: bool = True, quantize_acts: bool = True, dtype: torch.dtype = torch.bfloat16,
               routing: bool = False, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """The mixture-of-experts layer of mx_moe for any number of tokens (a prompt, a large batch): router, grouped
    products and weighted sum.  With quantize_acts x and silu(gate) * up go through MXFP4 (W4A4), else through bf16 (W4A16);
    what an expert gives a token is rounded to y's type before the weighted fp32 sum.

    In place of mx_moe: quantize_acts is True unless given, so that activations have four bits, which mx_moe's never have;
    quantize_acts=False keeps them in bf16, and mx_moe, for up to 64 tokens, in fp32's bits.  mx_moe is the faster one up to about
    ten tokens.  Else arguments, layouts and returns are mx_moe's (a row with NaN or +inf has NaN weights)."""
    dev = x.device
    assert x.dtype is torch.bfloat16, f"x: bf16, not {x.dtype}"
    assert logits.dtype in (torch.float32, torch.bfloat16), f"logits: fp32 or bf16, not {logits.dtype}"
    ld_x, ld_l = _rows(x, "x", w_gate_up.shape[1]), _rows(logits, "logits")
    t, h = x.shape
    assert logits.shape[0] == t, f"logits: {logits.shape[0]} rows, expected {t}"
    assert logits.device == dev and w_gate_up.codes.device == dev and w_down.codes.device == dev, "one device per call"
    out, ld_y, dt = _out(out, t, h, dtype, dev, "out")
    ids = weights = None
    if routing:
        ids = torch.empty((t, top_k), dtype=torch.int32, device=dev)
        weights = torch.empty((t, top_k), dtype=torch.float32, device=dev)
    e = logits.shape[1]
    if workspace is None:
        workspace = mx_experts_workspace(t, e, top_k, w_gate_up, w_down, quantize_acts, out.dtype)
    _call("mxfp4_experts", dev, x.data_ptr(), t, ld_x, logits.data_ptr(), _DT[logits.dtype], ld_l, e, top_k,
          1 if renormalize else 0, 1 if quantize_acts else 0, ctypes.byref(w_gate_up.c()), ctypes.byref(w_down.c()),
          out.data_ptr(), dt, ld_y, _opt(ids, dev, "ids"), _opt(weights, dev, "weights"), _opt(workspace, dev, "workspace"),
          _nbytes(workspace))
    return (out, ids, weights) if routing else out


@functools.lru_cache(maxsize=256)
def _adapters_size(device: int, *args) -> int:
    """Bytes of a workspace, which are planned for the current device.  (A call into the library takes as long as the rest of
    the binding's checks.)"""
    if device == _current_device():
        return int(load_library().mxfp4_adapters_workspace_size(*args))
    with torch.cuda.device(device):
        return int(load_library().mxfp4_adapters_workspace_size(*args))


def mx_adapters_workspace(m: int, w: MXFP4Tensor, adapters: int, rank: int, quantized_acts: bool = False) -> torch.Tensor | None:
    """A workspace for mx_gemm_adapters with m rows (None when it needs none).  Its contents do not matter; calls that share one
    must be ordered (same stream, or events)."""
    dev = w.codes.device
    n, k = w.shape
    return _workspace(_adapters_size(dev.index, m, n, k, adapters, rank, 1 if quantized_acts else 0), dev)


def mx_gemm_adapters(a: torch.Tensor, w: MXFP4Tensor, down: torch.Tensor, up: torch.Tensor, index: torch.Tensor,
                     scales: torch.Tensor | None = None, a_q: MXFP4Tensor | None = None, dtype: torch.dtype = torch.float32,
                     out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """A projection that requests share, with low-rank adapters of their own: C[m] = A[m] . W^T + scales[i] (A[m] .
    down[i]^T) . up[i]^T with i = index[m] (int32 [M], any order; outside 0 .. adapters - 1: no adapter).

    a: bf16 [M, K]; a_q: its MXFP4 form, for a W4A4 product (the branch takes `a`); w [N, K]; down [adapters, rank, K] and up
    [adapters, N, rank] bf16, dense, rank a multiple of 8 up to 256; scales fp32 [adapters].  C fp32 or bf16, rounded once.  From 512 adapters
    on rows of different adapters in turn are several times slower than side by side (include/mxfp4.h)."""
    assert isinstance(w, MXFP4Tensor), "w: an MXFP4Tensor is required"
    n, k = w.shape
    dev = w.codes.device
    assert a.dtype is torch.bfloat16 and a.device == dev, f"a: a bf16 tensor on {dev} is required"
    lda, m = _rows(a, "a", k), a.shape[0]
    assert down.dim() == 3, f"down: [adapters, rank, K] is required, not {tuple(down.shape)}"
    count, rank = down.shape[0], down.shape[1]
    a_ct = None
    if a_q is not None:
        assert a_q.shape == (m, k) and a_q.codes.device == dev, f"a_q: {a_q.shape} on {a_q.codes.device}, expected {(m, k)} on {dev}"
        a_ct = ctypes.byref(a_q.c())
    down_ptr = _words(down, "down", dev, torch.bfloat16, count, rank, k)
    up_ptr = _words(up, "up", dev, torch.bfloat16, count, n, rank)
    index_ptr = _words(index, "index", dev, torch.int32, m)
    scales_ptr = None if scales is None else _words(scales, "scales", dev, torch.float32, count)
    out, ldc, dt = _out(out, m, n, dtype, dev, "out")
    if workspace is None:
        workspace = mx_adapters_workspace(m, w, count, rank, a_q is not None)
    _call("mxfp4_gemm_adapters", dev, a.data_ptr(), a_ct, m, lda, ctypes.byref(w.c()), index_ptr, count, rank, down_ptr, up_ptr,
          scales_ptr, out.data_ptr(), dt, ldc, _opt(workspace, dev, "workspace"), _nbytes(workspace))
    return out
