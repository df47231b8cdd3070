"""One MoE layer of a residual stream, forward and backward, over the layer
operators: run on a GPU with

    python examples/moe_layer.py [--tokens 512] [--steps 3]

The layer's path, as a training step takes it on one GPU:

  norm      h = x + residual; rms_norm(h) in MXFP8 for the experts and in bf16
            for the router
  route     softmax of the router's logits, the topk experts of each token and
            their weights
  dispatch  the pairs sorted by expert, and the tokens' 8-bit rows written in
            that order (what an expert-parallel job would send)
  experts   each expert's run of rows through its weight, bf16 (torch matmul)
  combine   the expert rows weighted by the router and summed per token

Backward runs the same path the other way, straight through the 8-bit
rounding, and the gradients are clipped to a global norm before the update.  The
experts' products here stand in for whatever computes them; the rest is the
library.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import dequantize_reduce_transfer_amd as fq  # noqa: E402


class Norm(torch.autograd.Function):
    """(MXFP8 codes, E8M0 scales, h, y): the codes and scales carry no
    gradient of their own; the rows' gradient arrives at y."""

    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        out = fq.mx8_rms_norm_quantize(x, weight, eps, residual=residual, want_y=True, want_rstd=True)
        ctx.save_for_backward(out.h, weight, out.rstd)
        ctx.mark_non_differentiable(out.q, out.scales)
        return out.q, out.scales, out.h, out.y

    @staticmethod
    def backward(ctx, _q, _scales, dh, dy):
        h, weight, rstd = ctx.saved_tensors
        dx, dw = fq.fp8q_rms_norm_backward(dy.contiguous(), h, weight, rstd, dh=dh.contiguous())
        return dx, dx, dw.to(weight.dtype), None


class Route(torch.autograd.Function):
    """(weights, ids) of each token's topk experts; the choice has no gradient."""

    @staticmethod
    def forward(ctx, logits, topk):
        weights, ids = fq.fp8q_moe_route(logits, topk, normalize=False)
        ctx.save_for_backward(logits, weights, ids)
        ctx.mark_non_differentiable(ids)
        return weights, ids

    @staticmethod
    def backward(ctx, dweights, _ids):
        return fq.fp8q_moe_route_backward(dweights.contiguous(), *ctx.saved_tensors, normalize=False), None


class Dispatch(torch.autograd.Function):
    """The tokens' 8-bit rows at their experts, as bf16 values.  `y` is the
    rows' bf16 form, whose gradient this returns: the sum over a token's rows
    (a combine with weights of one)."""

    @staticmethod
    def forward(ctx, y, q, scales, slots):
        rows = torch.zeros(slots.numel(), q.shape[1], dtype=torch.uint8, device=q.device)
        rows_scales = torch.zeros(slots.numel(), scales.shape[1], dtype=torch.uint8, device=q.device)
        fq.fp8q_moe_permute(q, slots, scales=scales, out=rows, scales_out=rows_scales)
        ctx.save_for_backward(slots)
        return fq.mx8_dequantize(rows, rows_scales, out_dtype=torch.bfloat16)

    @staticmethod
    def backward(ctx, drows):
        (slots,) = ctx.saved_tensors
        return fq.fp8q_moe_combine(drows.contiguous(), slots), None, None, None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, slots, weights):
        ctx.save_for_backward(rows, slots, weights)
        return fq.fp8q_moe_combine(rows, slots, weights)

    @staticmethod
    def backward(ctx, dy):
        rows, slots, weights = ctx.saved_tensors
        drows = torch.zeros_like(rows)                     # places past the last pair stay zero
        _, dweights = fq.fp8q_moe_combine_backward(dy.contiguous(), rows, slots, weights, drows_out=drows)
        return drows, None, dweights


class MoeLayer(torch.nn.Module):
    def __init__(self, hidden=256, experts=16, topk=4, eps=1e-6, device="cuda"):
        super().__init__()
        self.experts, self.topk, self.eps = experts, topk, eps
        self.norm = torch.nn.Parameter(torch.ones(hidden, device=device))
        self.router = torch.nn.Parameter(torch.randn(hidden, experts, device=device) * hidden ** -0.5)
        self.weights = torch.nn.Parameter(
            (torch.randn(experts, hidden, hidden, device=device) * hidden ** -0.5).to(torch.bfloat16))

    def forward(self, x, residual):
        """(layer output, new residual stream): [tokens, hidden] bf16 each."""
        q, scales, h, y = Norm.apply(x, residual, self.norm, self.eps)
        weights, ids = Route.apply(y.float() @ self.router, self.topk)
        slots, _, offsets = fq.fp8q_moe_sort(ids, self.experts)
        rows = Dispatch.apply(y, q, scales, slots)
        ends = offsets.tolist()                            # torch's matmul wants the runs on the host
        out = torch.cat([rows[ends[e]:ends[e + 1]] @ self.weights[e] for e in range(self.experts)])
        return Combine.apply(out, slots, weights), h


def main(argv=None):
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--hidden", type=int, default=256)
    p.add_argument("--steps", type=int, default=3)
    p.add_argument("--max-norm", type=float, default=1.0)
    a = p.parse_args(argv)
    torch.manual_seed(0)
    layer = MoeLayer(a.hidden)
    optimizer = torch.optim.SGD(layer.parameters(), lr=0.5)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    residual = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    target = torch.randn(a.tokens, a.hidden, device="cuda")
    losses = []
    for step in range(a.steps):
        out, h = layer(x, residual)
        loss = (out.float() + h.float() - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        grads = [w.grad for w in layer.parameters()]
        sumsq = fq.fp8q_grad_sumsq(grads)                  # a sharded job adds it up over its ranks here
        norm = fq.fp8q_grad_clip(grads, sumsq, a.max_norm)
        optimizer.step()
        losses.append(float(loss.detach()))
        print("step %d loss %.5f gradient norm %.4f" % (step, losses[-1], float(norm)), flush=True)
    return losses


if __name__ == "__main__":
    main()
