"""The cases that the model's operators are timed on (perf/more_operators.py),
and drawn ones of the same ranges, against that file's own 64-bit forms.  Ids
are equal; the rest is within bounds of the outputs' types."""
import random

import pytest
import torch

from gpu_util import require_gpu
from layer_ref import TINY16, U16, U32
from perf import more_operators as cases

pytestmark = pytest.mark.gpu

CASES = [pytest.param(c, id=c["name"].replace(" ", "-")) for c in cases.listed()]
CASES += [pytest.param(cases.draw(random.Random(seed)), id="drawn-%d" % seed) for seed in range(24)]


def within(got, want, limit, what):
    worst = float(((got.double() - want).abs() - limit).max()) if got.numel() else 0.0
    assert worst <= 0.0, "%s: %.3g past its bound" % (what, worst)


def check_route(case, state, got, want):
    assert torch.equal(got["ids"].long(), want["ids"].long())
    # logits are within 30 of their row's largest: exp's argument and exp itself,
    # and a sum over at most 512 of them
    within(got["weights"], want["weights"], 600 * U32 * want["weights"], "weights")


def check_route_grad(case, state, got, want):
    mag = (state["weights"] * state["dweights"]).double().abs()
    mag = torch.where(state["ids"] >= 0, mag, 0.0).sum(1, keepdim=True)
    limit = 600 * U32 * (mag + want.abs())
    within(got, want, limit + (U16 * want.abs() + TINY16 if case["dtype"] == "bf16" else 0.0), "dlogits")


def check_experts(case, state, got, want):
    """bf16's own rounding, and what sums of fp32 products and h's 16 bits may
    add: 2^-11 of a row's largest value (a fp32 sum of n random products is off by
    about sqrt(n) * 2^-24 of their root of squares)."""
    within(got, want, U16 * want.abs() + 2.0 ** -11 * want.abs().amax(1, keepdim=True), "y")


def check_grad_norm(case, state, got, want):
    for a, b in zip(got, want):
        within(a, b, (case["elems"] + 2) * 2.0 ** -53 * b, "sum of squares")


def check_grad_clip(case, state, got, want):
    within(got["norm"], want["norm"], U32 * want["norm"], "norm")
    for a, b in zip(got["grads"], want["grads"]):
        within(a, b, (U16 if a.dtype == torch.bfloat16 else 0.0) * b.abs() + 3 * U32 * b.abs() + 2.0 ** -133, "gradient")


@pytest.mark.parametrize("case", CASES)
def test_case(case, monkeypatch):
    require_gpu()
    state = cases.prepare(case, 11)
    monkeypatch.setattr(cases, "own", True)
    got = cases.run(state)
    torch.cuda.synchronize()
    want = cases.exact(case, 11)
    {"route": check_route, "route_grad": check_route_grad, "experts": check_experts, "grad_norm": check_grad_norm,
     "grad_clip": check_grad_clip}[case["op"]](case, state, got, want)
