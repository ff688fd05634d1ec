"""MXFP4 (E2M1 codes, one power-of-two E8M0 scale per 32 elements of a row): quantization, expansion,
the product with MXFP4 weights and the mixture-of-experts layer for a few tokens.

A thin ctypes binding over the entry points of ``include/mxfp4.h``; the package re-exports its names.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import (_DT, _I32, _I64, _P, _SIGNATURES, _RESTYPES, _SZ, _check, _rows, _workspace, check_flags,
               load_library)

MX_OP_GEMM_BF16, MX_OP_GEMM_MX, MX_OP_MOE = 0, 1, 2
MX_BLOCK = 32
SKINNY_MAX_M = 16  # products of up to this many rows take no workspace
MOE_MAX_TOKENS, MOE_MAX_EXPERTS, MOE_MAX_TOP_K = 64, 512, 16
MX_EXPORTED = ["mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_moe", "mxfp4_workspace_size"]


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
})
_RESTYPES["mxfp4_workspace_size"] = _SZ


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
