"""The MoE layer's activation path: Python functions over ``libfp8q_layer.so``.

The residual stream's rows are normed straight into 8 bits, sent to their
experts in the codec's formats, and brought back; the gradients that training
needs are entry points of their own.  The C ABI and the formulas are in
``include/fp8q_layer.h``.  As with the codec's functions, tensors are checked
(a TypeError or ValueError), outputs and workspaces are allocated with torch
when the caller gives none, calls run on the current stream or on ``stream=``
(and allocate from that stream's memory), and a non-zero status raises
:class:`Fp8qError`; there is no CPU fallback.  The checks and allocations are
in ``csrc/layer_binding.cpp``.

Outputs carry no autograd history, also where an input requires a gradient: the
gradients are the ``..._backward`` functions (and a combine without weights, for
a permute's).  ``examples/moe_layer.py`` has the ``torch.autograd.Function``s
that tie them together.

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
import importlib.util
import os
from typing import NamedTuple, Optional

import torch

from . import BLOCK, E4M3, OUT_BF16, _check, _out_code

NORM_MAX_HIDDEN = 32768
MAX_HIDDEN = 1 << 20
MAX_TOPK = 64
MAX_EXPERTS = 1024

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8q_layer.so")
BINDING_PATH = os.path.join(_PKG, "_layer.so")
_lib = None
_native = None

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


def layer_lib(path: str = LIB_PATH) -> ctypes.CDLL:
    """``libfp8q_layer.so`` itself, its C ABI with argument types set (raises
    if unbuilt).  ``path`` names another build of it."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libfp8q_layer.so is not built (%s); run "
                           "`python -m dequantize_reduce_transfer_amd.build`" % path)
    L = ctypes.CDLL(path)
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
    if path == LIB_PATH:
        _lib = L
    return L


def _binding():
    """The module ``_layer.so`` (raises if unbuilt)."""
    global _native
    if _native is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError("_layer.so is not built (%s); run "
                               "`python -m dequantize_reduce_transfer_amd.build`" % BINDING_PATH)
        spec = importlib.util.spec_from_file_location(__package__ + "._layer", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native = module
    return _native


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _current(t) -> int:
    """The raw handle of the current stream of t's GPU (0 where t is not on
    one: the call is refused for that)."""
    if not (isinstance(t, torch.Tensor) and t.is_cuda):
        return 0
    if _raw_stream is not None:             # 0.1 us, against 2 for a Stream object
        return _raw_stream(t.get_device())
    return int(torch.cuda.current_stream(t.device).cuda_stream)


def _outputs(what: str, result):
    """The outputs of the binding's (status, outputs...)."""
    if result[0]:
        _check(result[0], what)
    return result[1:]


def _tensors(values):
    """The tensors among the values, and in lists and tuples of them."""
    for v in values:
        if isinstance(v, torch.Tensor):
            yield v
        elif isinstance(v, (list, tuple)):
            yield from _tensors(v)


def _on_stream(stream, what: str, function, t, *args):
    """``function(t, *args)``, a call without a stream of its own, on the stream
    that the caller named: it is current for the call.

    Outputs and workspaces are allocated from the current stream's own memory,
    so no work queued on another stream still uses them.  Every tensor of the
    call is recorded on the named stream, so that memory of other streams is
    kept until it is done, and the outputs on the caller's, which is to read
    them and may release them before it has."""
    first = next(_tensors((t, args)), None)
    if first is not None and first.is_cuda and stream.device != first.device:
        raise ValueError("%s: the stream is on %s, the tensors on %s" % (what, stream.device, first.device))
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.device(stream.device):  # setting a stream makes its GPU current too
        torch.cuda.set_stream(stream)       # 3 us less than torch.cuda.stream
        try:
            result = function(t, *args)
        finally:
            torch.cuda.set_stream(caller)
    outputs = result if isinstance(result, tuple) else (result,)
    for x in _tensors((t, args, outputs)):
        x.record_stream(stream)
    for x in outputs:
        if x is not None:
            x.record_stream(caller)
    return result


def row_scales(hidden: int) -> int:
    """fp32 scales of one row: one per 128 elements, the last block partial."""
    return (hidden + BLOCK - 1) // BLOCK


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
    Not tracked by autograd: :func:`fp8q_rms_norm_backward` is the gradient.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_rms_norm_quantize", fp8q_rms_norm_quantize, x, weight, eps, residual,
                          fmt, want_h, want_y, want_rstd, h_out, y_out, q_out, scales_out, rstd_out)
    return RmsNorm._make(_outputs("fp8q_rms_norm_quantize", (_native or _binding()).rms_norm_quantize(
        False, x, weight, eps, residual, fmt, want_h, want_y, want_rstd, h_out, y_out, q_out, scales_out,
        rstd_out, _current(x))))


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
    if stream is not None:
        return _on_stream(stream, "mx8_rms_norm_quantize", mx8_rms_norm_quantize, x, weight, eps, residual,
                          want_h, want_y, want_rstd, h_out, y_out, q_out, e8m0_out, rstd_out)
    return RmsNorm._make(_outputs("mx8_rms_norm_quantize", (_native or _binding()).rms_norm_quantize(
        True, x, weight, eps, residual, E4M3, want_h, want_y, want_rstd, h_out, y_out, q_out, e8m0_out,
        rstd_out, _current(x))))


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
    if stream is not None:
        return _on_stream(stream, "fp8q_rms_norm_backward", fp8q_rms_norm_backward, dy, h, weight, rstd, dh,
                          dx_out, dweight_out, workspace)
    return _outputs("fp8q_rms_norm_backward", (_native or _binding()).rms_norm_backward(
        dy, h, weight, rstd, dh, dx_out, dweight_out, workspace, _current(dy)))


def fp8q_rms_norm_backward_workspace(rows: int, hidden: int) -> int:
    """Bytes of workspace a norm's backward pass needs."""
    return int(layer_lib().fp8q_rms_norm_backward_workspace(rows, hidden))


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
    if stream is not None:
        return _on_stream(stream, "fp8q_moe_sort", fp8q_moe_sort, ids, experts, slots_out, pairs_out,
                          offsets_out, workspace)
    return _outputs("fp8q_moe_sort", (_native or _binding()).moe_sort(
        ids, experts, slots_out, pairs_out, offsets_out, workspace, _current(ids)))


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
    left as they are, slots outside the buffer are skipped.  Not tracked by
    autograd: :func:`fp8q_moe_combine` without weights is the gradient.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_moe_permute", fp8q_moe_permute, x, slots, scales, out, scales_out)
    return _outputs("fp8q_moe_permute", (_native or _binding()).moe_permute(
        x, slots, scales, out, scales_out, _current(x)))


def fp8q_moe_combine(rows: torch.Tensor, slots: torch.Tensor, weights: Optional[torch.Tensor] = None,
                     scales: Optional[torch.Tensor] = None, fmt: int = E4M3,
                     out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None):
    """Sum of each token's expert rows, weighted -> [tokens, hidden].

    rows [n, hidden]: bf16, or uint8 codes with their ``scales``: fp32
    [n, ceil(hidden / 128)] (``fmt`` E4M3 or E5M2), or uint8 E8M0
    [n, hidden / 32] (MXFP8).  weights fp32 [tokens, topk]; None sums the rows
    as they are, which for bf16 rows is the gradient of a permute.  Not tracked
    by autograd: :func:`fp8q_moe_combine_backward` is the gradient, of bf16 rows.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_moe_combine", fp8q_moe_combine, rows, slots, weights, scales, fmt,
                          out_dtype, out)
    return _outputs("fp8q_moe_combine", (_native or _binding()).moe_combine(
        rows, slots, weights, scales, fmt, _out_code(out_dtype) == OUT_BF16, out, _current(rows)))[0]


def fp8q_moe_combine_backward(dy: torch.Tensor, rows: torch.Tensor, slots: torch.Tensor,
                              weights: torch.Tensor, drows_out: Optional[torch.Tensor] = None,
                              dweights_out: Optional[torch.Tensor] = None, stream=None):
    """Gradients of a combine over bf16 rows -> (drows bf16 [n, hidden],
    dweights fp32 [tokens, topk]).  Rows of drows that no slot names are left
    as they are (an allocated one holds anything there).  Rows that were combined
    from codes are dequantized for it first."""
    if stream is not None:
        return _on_stream(stream, "fp8q_moe_combine_backward", fp8q_moe_combine_backward, dy, rows, slots,
                          weights, drows_out, dweights_out)
    return _outputs("fp8q_moe_combine_backward", (_native or _binding()).moe_combine_backward(
        dy, rows, slots, weights, drows_out, dweights_out, _current(dy)))
