"""MXFP4 (E2M1 codes, one power-of-two E8M0 scale per 32 elements of a row): quantization, expansion,
the product with MXFP4 weights and the mixture-of-experts layer for a few tokens.

A thin ctypes binding over the entry points of ``include/mxfp4.h``; the package re-exports its names.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch

from . import (_DT, _I32, _I64, _P, _SIGNATURES, _RESTYPES, _SZ, NVFP4Tensor, _check, _ptr, _rows, _stream, _workspace,
               check_flags, load_library)

MX_OP_GEMM_BF16, MX_OP_GEMM_MX, MX_OP_MOE = 0, 1, 2
MX_BLOCK = 32
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
        r, c = self.shape
        assert c % MX_BLOCK == 0 and tuple(self.scales.shape) == (r, c // MX_BLOCK), \
            f"MXFP4 scales: shape {tuple(self.scales.shape)}, expected {(r, c // MX_BLOCK)}"
        for t in (self.codes, self.scales):
            assert t.is_cuda and t.dtype == torch.uint8 and t.device == self.codes.device, \
                "MXFP4 codes and scales must be uint8 device tensors on one device"
            assert t.is_contiguous(), "MXFP4 codes and scales must be dense"
        return CMXTensor(self.codes.data_ptr(), self.scales.data_ptr(), r, c)


def _on(device: torch.device):
    """Make `device` current for a call: the library launches on the current device."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _same_device(device: torch.device, **tensors) -> None:
    for name, t in tensors.items():
        assert t is None or (t.is_cuda and t.device == device), f"{name}: expected a tensor on {device}"


def _out(out: torch.Tensor | None, rows: int, cols: int, dtype: torch.dtype, device, what: str):
    """The output matrix (allocated when not given) and its row stride."""
    assert dtype in (torch.float32, torch.bfloat16), f"{what}: dtype {dtype} not offered"
    if out is None:
        return torch.empty((rows, cols), dtype=dtype, device=device), cols
    _same_device(device, **{what: out})
    assert out.dtype == dtype and out.shape[0] == rows, f"{what}: {tuple(out.shape)} {out.dtype}"
    return out, _rows(out, what, cols)


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
    if out is None:
        out = MXFP4Tensor.empty(rows, cols, x.device)
    assert out.shape == (rows, cols), f"out: shape {out.shape}, expected {(rows, cols)}"
    if flags is None and check:
        flags = torch.zeros(1, dtype=torch.int32, device=x.device)
    _same_device(x.device, src_scale=src_scale, flags=flags, out=out.codes)
    assert src_scale is None or src_scale.dtype == torch.float32
    assert flags is None or flags.dtype == torch.int32
    ct = out.c()
    with _on(x.device):
        st = load_library().mxfp4_quantize(_ptr(x), _DT[x.dtype], ld, _ptr(src_scale), ctypes.byref(ct), _ptr(flags),
                                           _stream(x.device))
    _check(st, "mxfp4_quantize")
    out.flags = flags
    if check:
        check_flags(flags, "mxfp4_quantize")
    return out


def mx_dequantize(q: MXFP4Tensor, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None) -> torch.Tensor:
    """Expand MXFP4 to bf16 or fp32 (exact)."""
    rows, cols = q.shape
    dev = q.codes.device
    out, ld = _out(out, rows, cols, dtype if out is None else out.dtype, dev, "out")
    ct = q.c()
    with _on(dev):
        st = load_library().mxfp4_dequantize(ctypes.byref(ct), _ptr(out), _DT[out.dtype], ld, _stream(dev))
    _check(st, "mxfp4_dequantize")
    return out


def mx_gemm_workspace(a: torch.Tensor | MXFP4Tensor, w: MXFP4Tensor) -> torch.Tensor | None:
    """A workspace for mx_gemm(a, w), for callers that keep one (None when the product needs none).  Its
    contents do not matter; calls that share one must be ordered (same stream, or events)."""
    op = MX_OP_GEMM_MX if isinstance(a, MXFP4Tensor) else MX_OP_GEMM_BF16
    return _workspace(mx_workspace_size(op, a.shape[0], w.shape[0], w.shape[1]), w.codes.device)


def mx_gemm(a: torch.Tensor | MXFP4Tensor, w: MXFP4Tensor, dtype: torch.dtype = torch.float32,
            out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """C [M, N] (fp32 or bf16) = A . W^T with MXFP4 weights [N, K].  `a` is an MXFP4Tensor [M, K] (W4A4: FP4
    matrix instructions) or a bf16 tensor [M, K] (W4A16).  fp32 sums, rounded once."""
    assert isinstance(w, MXFP4Tensor), "w: an MXFP4Tensor is required"
    assert not isinstance(a, NVFP4Tensor), "a: NVFP4 activations do not go with MXFP4 weights"
    n, k = w.shape
    dev = w.codes.device
    m = a.shape[0]
    if isinstance(a, MXFP4Tensor):
        assert a.shape[1] == k, f"a: {a.shape[1]} columns, expected {k}"
        _same_device(dev, a=a.codes)
        a_ct, a_ptr, lda = ctypes.byref(a.c()), None, k
    else:
        assert a.dtype == torch.bfloat16, f"a: bf16 or MXFP4, not {a.dtype}"
        _same_device(dev, a=a)
        lda = _rows(a, "a", k)
        a_ct, a_ptr = None, _ptr(a)
    out, ldc = _out(out, m, n, dtype if out is None else out.dtype, dev, "out")
    wct = w.c()
    lib = load_library()
    with _on(dev):
        if workspace is None:
            workspace = mx_gemm_workspace(a, w)
        _same_device(dev, workspace=workspace)
        st = lib.mxfp4_gemm(a_ptr, a_ct, m, lda, ctypes.byref(wct), _ptr(out), _DT[out.dtype], ldc, _ptr(workspace),
                            0 if workspace is None else workspace.numel() * workspace.element_size(), _stream(dev))
    _check(st, "mxfp4_gemm")
    return out


def mx_moe_workspace(tokens: int, top_k: int, w_down: MXFP4Tensor) -> torch.Tensor | None:
    """A workspace for mx_moe (None without tokens).  Its contents do not matter; calls that share one
    must be ordered (same stream, or events)."""
    return _workspace(mx_workspace_size(MX_OP_MOE, tokens, top_k, w_down.shape[1]), w_down.codes.device)


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
    assert x.dtype == torch.bfloat16, f"x: bf16, not {x.dtype}"
    assert logits.dtype in (torch.float32, torch.bfloat16), f"logits: fp32 or bf16, not {logits.dtype}"
    ld_x, ld_l = _rows(x, "x", w_gate_up.shape[1]), _rows(logits, "logits")
    t, h = x.shape
    assert logits.shape[0] == t, f"logits: {logits.shape[0]} rows, expected {t}"
    _same_device(dev, logits=logits, w_gate_up=w_gate_up.codes, w_down=w_down.codes)
    out, ld_y = _out(out, t, h, dtype if out is None else out.dtype, dev, "out")
    ids = weights = None
    if routing:
        ids = torch.empty((t, top_k), dtype=torch.int32, device=dev)
        weights = torch.empty((t, top_k), dtype=torch.float32, device=dev)
    gct, dct = w_gate_up.c(), w_down.c()
    with _on(dev):
        if workspace is None:
            workspace = mx_moe_workspace(t, top_k, w_down)
        _same_device(dev, workspace=workspace)
        st = load_library().mxfp4_moe(_ptr(x), t, ld_x, _ptr(logits), _DT[logits.dtype], ld_l, logits.shape[1], top_k,
                                      1 if renormalize else 0, ctypes.byref(gct), ctypes.byref(dct), _ptr(out),
                                      _DT[out.dtype], ld_y, _ptr(ids), _ptr(weights), _ptr(workspace),
                                      0 if workspace is None else workspace.numel() * workspace.element_size(),
                                      _stream(dev))
    _check(st, "mxfp4_moe")
    return (out, ids, weights) if routing else out
