"""Python binding of ``libfp8q_layer.so``: the MoE layer's activation path.

The residual stream's rows are normed straight into 8 bits, sent to their
experts in the codec's formats, and brought back; the gradients that training
needs are entry points of their own.  The C ABI and the formulas are in
``include/fp8q_layer.h``; these functions, like the codec's in the package
itself, check tensors, allocate outputs and workspaces with torch when the
caller gives none, and pass raw pointers and a HIP stream.

  fp8q_rms_norm_quantize(x, weight, eps)      -> RmsNorm(q, scales, h, y, rstd)
  mx8_rms_norm_quantize(x, weight, eps)       -> RmsNorm(q, scales, h, y, rstd)
  fp8q_rms_norm_backward(dy, h, weight, rstd) -> (dx bf16, dweight f32 [hidden])
  fp8q_moe_sort(ids, experts)                 -> (slots, pairs, offsets), int32
  fp8q_moe_permute(x, slots)                  -> (rows, scales or None)
  fp8q_moe_combine(rows, slots, weights)      -> y f32 or bf16 [tokens, hidden]
  fp8q_moe_combine_backward(dy, rows, slots, weights)
                                              -> (drows bf16, dweights f32)
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

from . import (BLOCK, E4M3, MX_BLOCK, _fmt, _need, _out_code, _run, _stream)

ROWS_BF16 = 0
ROWS_E4M3 = 1
ROWS_E5M2 = 2
ROWS_MX8 = 3
NORM_MAX_HIDDEN = 32768
MAX_TOPK = 64
MAX_EXPERTS = 1024

_PKG = os.path.dirname(os.path.abspath(__file__))
# FP8Q_LAYER_LIB selects another build of the same library.
LIB_PATH = os.environ.get("FP8Q_LAYER_LIB") or os.path.join(_PKG, "libfp8q_layer.so")
_lib = None

EXPORTS = ("fp8q_rms_norm_quantize", "mx8_rms_norm_quantize", "fp8q_rms_norm_backward_workspace",
           "fp8q_rms_norm_backward", "fp8q_moe_sort_workspace", "fp8q_moe_sort",
           "fp8q_moe_permute", "fp8q_moe_combine", "fp8q_moe_combine_backward")


class RmsNorm(NamedTuple):
    """What a norm returns: 8-bit rows and their scales (fp32, or E8M0 bytes),
    and, where asked for, the rounded sum h, the normed rows in bf16 and each
    row's 1/rms."""

    q: torch.Tensor
    scales: torch.Tensor
    h: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


def layer_lib() -> ctypes.CDLL:
    """The loaded ``libfp8q_layer.so`` with argument types set (raises if unbuilt)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError("libfp8q_layer.so is not built (%s); run "
                           "`python -m dequantize_reduce_transfer_amd.build`" % LIB_PATH)
    L = ctypes.CDLL(LIB_PATH)
    P, S, I, F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
    L.fp8q_rms_norm_quantize.argtypes = [P, P, P, I, F, S, S, I, P, P, P, P, P, P]
    L.mx8_rms_norm_quantize.argtypes = [P, P, P, I, F, S, S, P, P, P, P, P, P]
    L.fp8q_rms_norm_backward_workspace.argtypes = [S, S]
    L.fp8q_rms_norm_backward.argtypes = [P, P, P, I, P, P, S, S, P, P, P, S, P]
    L.fp8q_moe_sort_workspace.argtypes = [S, I, I]
    L.fp8q_moe_sort.argtypes = [P, I, S, I, I, P, P, P, P, S, P]
    L.fp8q_moe_permute.argtypes = [P, S, P, S, P, S, I, S, P, P, P]
    L.fp8q_moe_combine.argtypes = [P, I, P, P, P, S, I, S, S, P, I, P]
    L.fp8q_moe_combine_backward.argtypes = [P, P, P, P, S, I, S, S, P, P, P]
    for name in EXPORTS:
        getattr(L, name).restype = S if name.endswith("_workspace") else I
    _lib = L
    return L


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _given(*tensors):
    return [t for t in tensors if t is not None]


def _rows(t: torch.Tensor, name: str):
    """(rows, hidden) of a tensor whose last dimension is the row."""
    if t.dim() < 1:
        raise ValueError("%s needs at least one dimension" % name)
    hidden = t.shape[-1]
    return (t.numel() // hidden if hidden else 0), hidden


def _weight(w: torch.Tensor, hidden: int) -> int:
    if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("weight must be a float32 or bfloat16 tensor")
    _need(w, w.dtype, "weight")
    if w.numel() != hidden:
        raise ValueError("weight must hold hidden = %d values" % hidden)
    return 0 if w.dtype == torch.float32 else 1


def _shaped(t: Optional[torch.Tensor], shape, dtype, device, name: str) -> torch.Tensor:
    """The caller's output, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be of shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def row_scales(hidden: int) -> int:
    """fp32 scales of one row: one per 128 elements, the last block partial."""
    return (hidden + BLOCK - 1) // BLOCK


def _norm(what, mx, fmt, x, weight, eps, residual, want_h, want_y, want_rstd, h_out, y_out, q_out,
          scales_out, rstd_out, stream):
    _need(x, torch.bfloat16, "x")
    rows, hidden = _rows(x, "x")
    wcode = _weight(weight, hidden)
    if residual is not None:
        _need(residual, torch.bfloat16, "residual")
        if residual.shape != x.shape:
            raise ValueError("residual must have the shape of x")
    elif h_out is not None:
        raise ValueError("h_out needs a residual: without one h is x")
    if mx and hidden % MX_BLOCK:
        raise ValueError("hidden must be a multiple of 32")
    dev = x.device
    h = _shaped(h_out, x.shape, torch.bfloat16, dev, "h_out") \
        if residual is not None and (want_h or h_out is not None) else None
    y = _shaped(y_out, x.shape, torch.bfloat16, dev, "y_out") if want_y or y_out is not None else None
    rstd = _shaped(rstd_out, x.shape[:-1], torch.float32, dev, "rstd_out") \
        if want_rstd or rstd_out is not None else None
    q = _shaped(q_out, x.shape, torch.uint8, dev, "q_out")
    if mx:
        scales = _shaped(scales_out, (rows, hidden // MX_BLOCK), torch.uint8, dev, "e8m0_out")
    else:
        scales = _shaped(scales_out, (rows, row_scales(hidden)), torch.float32, dev, "scales_out")
    args = [x.data_ptr(), _ptr(residual), weight.data_ptr(), wcode, float(eps), rows, hidden]
    if not mx:
        args.append(_fmt(fmt))
    fn = layer_lib().mx8_rms_norm_quantize if mx else layer_lib().fp8q_rms_norm_quantize
    _run(what, _given(x, residual, weight, h, y, q, scales, rstd), fn, *args, _ptr(h), _ptr(y),
         q.data_ptr(), scales.data_ptr(), _ptr(rstd), _stream(x, stream), stream=stream)
    return RmsNorm(q, scales, h, y, rstd)


def fp8q_rms_norm_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                           residual: Optional[torch.Tensor] = None, fmt: int = E4M3,
                           want_h: bool = True, want_y: bool = False, want_rstd: bool = False,
                           h_out: Optional[torch.Tensor] = None,
                           y_out: Optional[torch.Tensor] = None,
                           q_out: Optional[torch.Tensor] = None,
                           scales_out: Optional[torch.Tensor] = None,
                           rstd_out: Optional[torch.Tensor] = None, stream=None) -> RmsNorm:
    """rms_norm(x + residual) * weight as FP8 rows with an fp32 scale per 128.

    x, residual bf16 [..., hidden]; weight fp32 or bf16 [hidden].  ``h`` (the
    sum in bf16; ``h_out`` may be x or residual itself) comes with a residual,
    ``y`` (the normed rows in bf16) and ``rstd`` (fp32 [...]) when asked for.
    """
    return _norm("fp8q_rms_norm_quantize", False, fmt, x, weight, eps, residual, want_h, want_y,
                 want_rstd, h_out, y_out, q_out, scales_out, rstd_out, stream)


def mx8_rms_norm_quantize(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6,
                          residual: Optional[torch.Tensor] = None, want_h: bool = True,
                          want_y: bool = False, want_rstd: bool = False,
                          h_out: Optional[torch.Tensor] = None,
                          y_out: Optional[torch.Tensor] = None,
                          q_out: Optional[torch.Tensor] = None,
                          e8m0_out: Optional[torch.Tensor] = None,
                          rstd_out: Optional[torch.Tensor] = None, stream=None) -> RmsNorm:
    """rms_norm(x + residual) * weight as MXFP8 rows (hidden a multiple of 32);
    otherwise as :func:`fp8q_rms_norm_quantize`."""
    return _norm("mx8_rms_norm_quantize", True, None, x, weight, eps, residual, want_h, want_y,
                 want_rstd, h_out, y_out, q_out, e8m0_out, rstd_out, stream)


def fp8q_rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                           rstd: torch.Tensor, dh: Optional[torch.Tensor] = None,
                           dx_out: Optional[torch.Tensor] = None,
                           dweight_out: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of a norm, straight through its 8-bit rounding -> (dx, dweight).

    dy: gradient of the normed rows, h: the forward's rows (bf16 [..., hidden]),
    rstd: the forward's fp32 [...], dh: gradient of the residual stream past
    the norm, added to dx.  dx (bf16) is the gradient of both x and the
    residual; ``dx_out`` may be dy or dh itself.  dweight is fp32 [hidden].
    ``workspace``: uint8, ``fp8q_rms_norm_backward_workspace`` bytes.
    """
    _need(dy, torch.bfloat16, "dy")
    _need(h, torch.bfloat16, "h")
    _need(rstd, torch.float32, "rstd")
    rows, hidden = _rows(h, "h")
    if dy.shape != h.shape or rstd.numel() != rows:
        raise ValueError("dy must have the shape of h, and rstd one value a row")
    if dh is not None:
        _need(dh, torch.bfloat16, "dh")
        if dh.shape != h.shape:
            raise ValueError("dh must have the shape of h")
    wcode = _weight(weight, hidden)
    dx = _shaped(dx_out, h.shape, torch.bfloat16, h.device, "dx_out")
    dw = _shaped(dweight_out, (hidden,), torch.float32, h.device, "dweight_out")
    L = layer_lib()
    ws, nbytes = _workspace(workspace, L.fp8q_rms_norm_backward_workspace(rows, hidden), h.device)
    _run("fp8q_rms_norm_backward", _given(dy, h, weight, rstd, dh, dx, dw, ws),
         L.fp8q_rms_norm_backward, dy.data_ptr(), h.data_ptr(), weight.data_ptr(), wcode,
         rstd.data_ptr(), _ptr(dh), rows, hidden, dx.data_ptr(), dw.data_ptr(), _ptr(ws), nbytes,
         _stream(h, stream), stream=stream)
    return dx, dw


def fp8q_rms_norm_backward_workspace(rows: int, hidden: int) -> int:
    """Bytes of workspace a norm's backward pass needs."""
    return int(layer_lib().fp8q_rms_norm_backward_workspace(rows, hidden))


def _workspace(given, nbytes: int, device):
    if given is None:
        return (torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None), nbytes
    _need(given, torch.uint8, "workspace")
    if given.numel() < nbytes:
        raise ValueError("workspace must hold %d bytes" % nbytes)
    return given, given.numel()


def _slots(slots: torch.Tensor, tokens: Optional[int] = None):
    """(tokens, topk) of a slot table."""
    _need(slots, torch.int32, "slots")
    if slots.dim() != 2:
        raise ValueError("slots must be [tokens, topk]")
    if tokens is not None and slots.shape[0] != tokens:
        raise ValueError("slots must have one row a token")
    if not 1 <= slots.shape[1] <= MAX_TOPK:
        raise ValueError("topk must be 1 .. %d" % MAX_TOPK)
    return slots.shape


def fp8q_moe_sort(ids: torch.Tensor, experts: int, slots_out: Optional[torch.Tensor] = None,
                  pairs_out: Optional[torch.Tensor] = None,
                  offsets_out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Pairs (token, choice) in stable order of their expert -> (slots, pairs, offsets).

    ids: int32 or int64 [tokens, topk]; an id outside [0, experts) has no
    place.  slots int32 [tokens, topk]: each pair's place, or -1; pairs int32
    [tokens * topk]: the pair at each place, -1 past the last; offsets int32
    [experts + 1]: each expert's first place, then their number.
    """
    if not isinstance(ids, torch.Tensor) or ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be an int32 or int64 tensor")
    _need(ids, ids.dtype, "ids")
    if ids.dim() != 2 or not 1 <= ids.shape[1] <= MAX_TOPK:
        raise ValueError("ids must be [tokens, topk], topk 1 .. %d" % MAX_TOPK)
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError("experts must be 1 .. %d" % MAX_EXPERTS)
    tokens, topk = ids.shape
    dev = ids.device
    slots = _shaped(slots_out, ids.shape, torch.int32, dev, "slots_out")
    pairs = _shaped(pairs_out, (tokens * topk,), torch.int32, dev, "pairs_out")
    offsets = _shaped(offsets_out, (experts + 1,), torch.int32, dev, "offsets_out")
    L = layer_lib()
    ws, nbytes = _workspace(workspace, L.fp8q_moe_sort_workspace(tokens, topk, experts), dev)
    _run("fp8q_moe_sort", _given(ids, slots, pairs, offsets, ws), L.fp8q_moe_sort, ids.data_ptr(),
         ids.element_size(), tokens, topk, experts, slots.data_ptr(), pairs.data_ptr(),
         offsets.data_ptr(), _ptr(ws), nbytes, _stream(ids, stream), stream=stream)
    return slots, pairs, offsets


def fp8q_moe_sort_workspace(tokens: int, topk: int, experts: int) -> int:
    """Bytes of workspace a sort needs."""
    return int(layer_lib().fp8q_moe_sort_workspace(tokens, topk, experts))


def fp8q_moe_permute(x: torch.Tensor, slots: torch.Tensor, scales: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, scales_out: Optional[torch.Tensor] = None,
                     stream=None):
    """Each token's row, and its scales, written to its places -> (rows, scales).

    x [tokens, hidden] of any dtype, scales [tokens, s] of any dtype or none;
    slots int32 [tokens, topk].  ``out`` [rows, hidden] (tokens * topk rows
    when allocated here) and ``scales_out`` [rows, s]: rows no slot names are
    left as they are, slots outside the buffer are skipped.
    """
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    _need(x, x.dtype, "x")
    if x.dim() != 2:
        raise ValueError("x must be [tokens, hidden]")
    tokens, topk = _slots(slots, x.shape[0])
    rows = tokens * topk if out is None else (out.shape[0] if out.dim() else 0)
    out = _shaped(out, (rows, x.shape[1]), x.dtype, x.device, "out")
    sbytes = 0
    if scales is not None:
        _need(scales, scales.dtype, "scales")
        if scales.dim() != 2 or scales.shape[0] != tokens:
            raise ValueError("scales must be [tokens, scales a row]")
        sbytes = scales.shape[1] * scales.element_size()
        scales_out = _shaped(scales_out, (rows, scales.shape[1]), scales.dtype, x.device, "scales_out")
    elif scales_out is not None:
        raise ValueError("scales_out needs scales")
    _run("fp8q_moe_permute", _given(x, slots, scales, out, scales_out),
         layer_lib().fp8q_moe_permute, x.data_ptr(), x.shape[1] * x.element_size(), _ptr(scales),
         sbytes, slots.data_ptr(), tokens, topk, rows, out.data_ptr(), _ptr(scales_out),
         _stream(x, stream), stream=stream)
    return out, scales_out


def fp8q_moe_combine(rows: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None,
                     scales: Optional[torch.Tensor] = None, fmt: int = E4M3,
                     out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None):
    """Sum of each token's expert rows, weighted -> [tokens, hidden].

    rows [n, hidden]: bf16, or uint8 codes with their ``scales``: fp32
    [n, ceil(hidden / 128)] (``fmt`` E4M3 or E5M2), or uint8 E8M0
    [n, hidden / 32] (MXFP8).  weights fp32 [tokens, topk]; None sums the rows
    as they are, which for bf16 rows is the gradient of a permute.
    """
    tokens, topk = _slots(slots)
    if not isinstance(rows, torch.Tensor) or rows.dtype not in (torch.bfloat16, torch.uint8):
        raise TypeError("rows must be a bfloat16 tensor, or uint8 codes")
    _need(rows, rows.dtype, "rows")
    if rows.dim() != 2:
        raise ValueError("rows must be [n, hidden]")
    n, hidden = rows.shape
    if rows.dtype == torch.bfloat16:
        if scales is not None:
            raise ValueError("bf16 rows have no scales")
        code = ROWS_BF16
    else:
        if not isinstance(scales, torch.Tensor) or scales.dtype not in (torch.float32, torch.uint8):
            raise TypeError("codes need scales: a float32 tensor, or uint8 E8M0 codes")
        _need(scales, scales.dtype, "scales")
        if scales.dtype == torch.uint8:
            if hidden % MX_BLOCK:
                raise ValueError("hidden must be a multiple of 32")
            code, each = ROWS_MX8, hidden // MX_BLOCK
        else:
            code, each = ROWS_E4M3 + _fmt(fmt), row_scales(hidden)
        if scales.numel() != n * each:
            raise ValueError("scales must hold %d values a row" % each)
    if weights is not None:
        _need(weights, torch.float32, "weights")
        if weights.shape != slots.shape:
            raise ValueError("weights must have the shape of slots")
    out = _shaped(out, (tokens, hidden), out_dtype, rows.device, "out")
    _run("fp8q_moe_combine", _given(rows, scales, slots, weights, out),
         layer_lib().fp8q_moe_combine, rows.data_ptr(), code, _ptr(scales), slots.data_ptr(),
         _ptr(weights), tokens, topk, n, hidden, out.data_ptr(), _out_code(out_dtype),
         _stream(rows, stream), stream=stream)
    return out


def fp8q_moe_combine_backward(dy: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor,
                              weights: torch.Tensor, drows_out: Optional[torch.Tensor] = None,
                              dweights_out: Optional[torch.Tensor] = None, stream=None):
    """Gradients of a combine over bf16 rows -> (drows bf16 [n, hidden],
    dweights fp32 [tokens, topk]).  Rows of drows that no slot names are left
    as they are (an allocated one holds anything there)."""
    _need(dy, torch.bfloat16, "dy")
    _need(rows, torch.bfloat16, "rows")
    if dy.dim() != 2 or rows.dim() != 2 or dy.shape[1] != rows.shape[1]:
        raise ValueError("dy must be [tokens, hidden] and rows [n, hidden]")
    tokens, topk = _slots(slots, dy.shape[0])
    _need(weights, torch.float32, "weights")
    if weights.shape != slots.shape:
        raise ValueError("weights must have the shape of slots")
    drows = _shaped(drows_out, rows.shape, torch.bfloat16, dy.device, "drows_out")
    dweights = _shaped(dweights_out, slots.shape, torch.float32, dy.device, "dweights_out")
    _run("fp8q_moe_combine_backward", _given(dy, rows, slots, weights, drows, dweights),
         layer_lib().fp8q_moe_combine_backward, dy.data_ptr(), rows.data_ptr(), slots.data_ptr(),
         weights.data_ptr(), tokens, topk, rows.shape[0], dy.shape[1], drows.data_ptr(),
         dweights.data_ptr(), _stream(dy, stream), stream=stream)
    return drows, dweights
