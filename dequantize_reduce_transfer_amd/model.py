"""The model's operators on both ends of the wire: Python functions over
``libfp8q_model.so``.

A receiver serves an MoE layer straight from weights in the codec's formats:
the routing, and the whole layer for a few tokens.  A trainer takes the
routing's gradient, and between the reduce and the update the norm of its
gradients and their clipping.  The C ABI and the formulas are in
``include/fp8q_model.h``; what holds of ``layer.py``'s functions (checks,
allocations, streams, errors, no autograd history, no CPU fallback) holds of
these.  The checks and allocations are in ``csrc/model_binding.cpp``.

  fp8q_moe_route(logits, topk)                -> (weights f32, ids int32) [tokens, topk]
  fp8q_moe_route_backward(dweights, logits, weights, ids) -> dlogits
  fp8q_moe_experts(x, ids, weights, gate, up, down)       -> y bf16 or f32 [tokens, hidden]
  fp8q_grad_sumsq(grads)                      -> sum of squares f64 [1]
  fp8q_grad_clip(grads, sumsq, max_norm)      -> norm f32 [1]; grads are scaled in place
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from typing import Optional, Sequence

import torch

from . import E4M3, OUT_BF16, _out_code
from .layer import _current, _on_stream, _outputs

EXPERTS_MAX_PAIRS = 1024
EXPERTS_MAX_SIZE = 65536

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8q_model.so")
BINDING_PATH = os.path.join(_PKG, "_model.so")
_lib = None
_native = None

EXPORTS = ("fp8q_moe_route", "fp8q_moe_route_backward", "fp8q_moe_experts_workspace", "fp8q_moe_experts",
           "fp8q_grad_sumsq_workspace", "fp8q_grad_sumsq", "fp8q_grad_clip")


class ExpertMatrix(ctypes.Structure):
    """``fp8q_expert_matrix``."""

    _fields_ = [("rows", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("expert_rows", ctypes.c_size_t)]


class Grad(ctypes.Structure):
    """``fp8q_grad``."""

    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("count", ctypes.c_size_t),
                ("scale_count", ctypes.c_size_t), ("dtype", ctypes.c_int)]


def model_lib(path: str = LIB_PATH) -> ctypes.CDLL:
    """``libfp8q_model.so`` itself, its C ABI with argument types set (raises
    if unbuilt).  ``path`` names another build of it."""
    global _lib
    if _lib is not None and path == LIB_PATH:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libfp8q_model.so is not built (%s); run "
                           "`python -m dequantize_reduce_transfer_amd.build`" % path)
    L = ctypes.CDLL(path)
    P, S, I, D = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_double
    M, G = ctypes.POINTER(ExpertMatrix), ctypes.POINTER(Grad)
    L.fp8q_moe_route.argtypes = [P, I, S, I, I, I, P, P, P]
    L.fp8q_moe_route_backward.argtypes = [P, P, I, P, P, S, I, I, I, P, P]
    L.fp8q_moe_experts_workspace.argtypes = [S, I, I, S, S, I]
    L.fp8q_moe_experts.argtypes = [P, P, I, P, I, M, M, M, S, I, I, S, S, P, I, P, S, P]
    L.fp8q_grad_sumsq_workspace.argtypes = [G, S]
    L.fp8q_grad_sumsq.argtypes = [G, S, P, P, S, P]
    L.fp8q_grad_clip.argtypes = [G, S, P, D, D, P, P]
    for name in EXPORTS:
        getattr(L, name).restype = S if name.endswith("_workspace") else I
    if path == LIB_PATH:
        _lib = L
    return L


def _binding():
    """The module ``_model.so`` (raises if unbuilt)."""
    global _native
    if _native is None:
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError("_model.so is not built (%s); run "
                               "`python -m dequantize_reduce_transfer_amd.build`" % BINDING_PATH)
        spec = importlib.util.spec_from_file_location(__package__ + "._model", BINDING_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _native = module
    return _native


def fp8q_moe_route(logits: torch.Tensor, topk: int, normalize: bool = True,
                   weights_out: Optional[torch.Tensor] = None, ids_out: Optional[torch.Tensor] = None,
                   stream=None):
    """Each token's ``topk`` experts and their softmax weights -> (weights, ids).

    logits fp32 or bf16 [tokens, experts]; ids int32 [tokens, topk], the largest
    logit's expert first, of equal ones the lowest; weights fp32 [tokens, topk],
    with ``normalize`` over the sum of the chosen ones.  An expert whose logit
    is -inf is never chosen: a token with fewer than ``topk`` others has ids of
    -1 and weights of 0 behind them, which the sort, the combine and the experts
    leave out.  A row that holds a NaN or +inf gets NaN weights.  Not tracked by
    autograd: :func:`fp8q_moe_route_backward` is the gradient.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_moe_route", fp8q_moe_route, logits, topk, normalize, weights_out, ids_out)
    return _outputs("fp8q_moe_route", (_native or _binding()).moe_route(
        logits, topk, normalize, weights_out, ids_out, _current(logits)))


def fp8q_moe_route_backward(dweights: torch.Tensor, logits: torch.Tensor, weights: torch.Tensor,
                            ids: torch.Tensor, normalize: bool = True,
                            dlogits_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Gradient of a routing's logits, of their dtype [tokens, experts].

    dweights: gradient of the weights (fp32 [tokens, topk]); logits, weights and
    ids as in the forward pass, whose ``normalize`` it takes too.  Entries whose
    id is outside the experts are left out.  ``dlogits_out`` may be ``logits``
    itself, and is changed in place to autograd.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_moe_route_backward", fp8q_moe_route_backward, dweights, logits, weights,
                          ids, normalize, dlogits_out)
    return _outputs("fp8q_moe_route_backward", (_native or _binding()).moe_route_backward(
        dweights, logits, weights, ids, normalize, dlogits_out, _current(dweights)))[0]


def fp8q_moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, gate: torch.Tensor,
                     up: torch.Tensor, down: torch.Tensor, gate_scales: Optional[torch.Tensor] = None,
                     up_scales: Optional[torch.Tensor] = None, down_scales: Optional[torch.Tensor] = None,
                     fmt: int = E4M3, out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A whole MoE layer for a few tokens -> [tokens, hidden]:
    ``sum_j weights[t, j] * down_e (silu(gate_e x_t) * (up_e x_t))`` with
    ``e = ids[t, j]``.

    x bf16 [tokens, hidden]; ids int32 or int64 and weights fp32 [tokens, topk],
    tokens * topk up to 1024; an id outside the experts (padding, or an expert
    that lives elsewhere) is left out.  gate and up [experts, inter, hidden],
    down [experts, hidden, inter]: bf16, or uint8 codes with their scales as the
    codec's quantize leaves them: fp32, one per 128 of a row (``fmt`` E4M3 or
    E5M2), or uint8 E8M0, one per 32 (MXFP8).  The experts may be any whole
    number of rows apart, so that gate and up may be halves of one [experts,
    2 * inter, hidden] tensor, and their scales (3-D then) of one as well.
    ``out_dtype`` bf16 or fp32 (to be added up over GPUs).  ``workspace``: uint8,
    :func:`fp8q_moe_experts_workspace` bytes.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_moe_experts", fp8q_moe_experts, x, ids, weights, gate, up, down,
                          gate_scales, up_scales, down_scales, fmt, out_dtype, out, workspace)
    return _outputs("fp8q_moe_experts", (_native or _binding()).moe_experts(
        x, ids, weights, gate, up, down, gate_scales, up_scales, down_scales, fmt,
        _out_code(out_dtype) == OUT_BF16, out, workspace, _current(x)))[0]


def fp8q_moe_experts_workspace(tokens: int, topk: int, experts: int, hidden: int, inter: int,
                               out_dtype=torch.bfloat16) -> int:
    """Bytes of workspace that :func:`fp8q_moe_experts` needs."""
    return int(model_lib().fp8q_moe_experts_workspace(tokens, topk, experts, hidden, inter, _out_code(out_dtype)))


def _first(grads, other):
    """The tensor whose GPU a list's call is on."""
    return grads[0] if isinstance(grads, (list, tuple)) and grads else other


def fp8q_grad_sumsq(grads: Sequence[torch.Tensor], scales: Optional[Sequence] = None, fmt: int = E4M3,
                    out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Sum of squares over a list of gradients -> fp64 [1].

    grads: fp32 or bf16 tensors, or uint8 codes of format ``fmt``, whose entry of
    ``scales`` (a list as long; None for the others) holds one fp32 scale per
    128 codes, or one.  Summed in fp64, in an order that the sizes fix.  Its
    square root is the global norm; over ranks that hold different gradients
    the sums add up (``all_reduce``) before :func:`fp8q_grad_clip`.
    ``workspace``: uint8; 16 KiB for every 160 gradients begun are always enough.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_grad_sumsq", fp8q_grad_sumsq, grads, scales, fmt, out, workspace)
    return _outputs("fp8q_grad_sumsq", (_native or _binding()).grad_sumsq(
        grads, scales, fmt, out, workspace, _current(_first(grads, out))))[0]


def fp8q_grad_clip(grads: Sequence[torch.Tensor], sumsq: torch.Tensor, max_norm: float,
                   scales: Optional[Sequence] = None, fmt: int = E4M3, eps: float = 1e-6,
                   norm_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Clips gradients in place to a largest global norm -> that norm, fp32 [1].

    grads, scales, fmt as in :func:`fp8q_grad_sumsq`, none overlapping another;
    sumsq fp64 [1], of the whole gradient.  Every gradient is multiplied by
    ``min(1, max_norm / (sqrt(sumsq) + eps))``; of codes, their scales are, and
    the codes stay.  Nothing is written where that is 1.  A NaN norm makes them
    all NaN.  To autograd the call is an in-place change of them (codes: of their
    scales), whatever the norm: a graph that has saved one refuses its backward.
    """
    if stream is not None:
        return _on_stream(stream, "fp8q_grad_clip", fp8q_grad_clip, grads, sumsq, max_norm, scales, fmt, eps,
                          norm_out)
    return _outputs("fp8q_grad_clip", (_native or _binding()).grad_clip(
        grads, sumsq, max_norm, scales, fmt, eps, norm_out, _current(sumsq)))[0]
