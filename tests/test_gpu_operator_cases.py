"""The cases that the layer operators are timed on (perf/operators.py), and
drawn ones of the same ranges, against that file's own 64-bit forms: the large
grids, whose workgroups take rows in another order than their own, among them.
Integers and copied bytes are equal; the rest is within the bounds that
test_gpu_rms_norm.py and test_gpu_moe.py derive."""
import random

import pytest
import torch

from gpu_util import require_gpu
from layer_ref import TINY16, U16, U32
from perf import operators

pytestmark = pytest.mark.gpu

RSTD = 32 * U32                        # 1/rms against 64 bits
NORMED = 40 * U32                      # the normed values: that, and their own roundings

CASES = [pytest.param(c, id=c["name"].replace(" ", "-")) for c in operators.listed()]
CASES += [pytest.param(operators.draw(random.Random(seed)), id="drawn-%d" % seed) for seed in range(24)]


def within(got, want, limit, what):
    worst = float(((got.double() - want).abs() - limit).max()) if got.numel() else 0.0
    assert worst <= 0.0, "%s: %.3g past its bound" % (what, worst)


def blocks(t, group):
    """Rows in blocks, the last filled up with zeros: [rows, blocks, group]."""
    count = -(-t.shape[1] // group)
    return torch.nn.functional.pad(t, (0, count * group - t.shape[1])).view(t.shape[0], count, group)


def check_norm(case, state, got, want):
    group = operators.GROUP[case["fmt"]]
    if case["residual"]:
        within(got["h"], want["h"], (U16 + 2 * U32) * want["h"].abs() + TINY16, "h")
    if case["y"]:
        within(got["y"], want["y"], (U16 + 2 * NORMED) * want["y"].abs() + TINY16, "y")
    if case["rstd"]:
        within(got["rstd"], want["rstd"], RSTD * want["rstd"], "rstd")
    q, q64 = blocks(got["q"].double(), group), blocks(want["q"], group)
    scales = got["scales"].double()
    # A code is its value's nearest: half a step off, 2^-4 (E5M2 2^-3) of it or
    # half the smallest one.  An fp32 scale has the values' error and its own.
    rel, least = (2.0 ** -3, 2.0 ** -17) if case["fmt"] == "e5m2" else (2.0 ** -4, 2.0 ** -10)
    if case["fmt"] == "mx8":
        # powers of two: equal, but where the block's largest value is one itself
        # to within its error (or, a step lower, saturates)
        ratio, top = scales / want["scales"], q64.abs().amax(2)
        assert ((ratio == 1) | ((ratio == 0.5) & (top <= 256 * (1 + NORMED))) | ((ratio == 2) & (top == 448))).all()
        same = (ratio == 1)[:, :, None]
        q, q64 = torch.where(same, q, 0.0), torch.where(same, q64, 0.0)
    else:
        within(scales, want["scales"], 2 * NORMED * want["scales"], "scales")
    within(q, q64, (rel + 3 * NORMED) * q64.abs() + least, "codes")


def check_norm_grad(case, state, got, want):
    h, w = state["h"].double(), state["w"].double()
    inv = state["inv"].double()[:, None]
    g = (state["dy"].double() * w).abs()
    mag = (g + h.abs() * inv * inv * (g * h.abs()).mean(1, keepdim=True)) * inv
    if case["residual"]:
        mag += state["dh"].double().abs()
    within(got["dx"], want["dx"], U16 * want["dx"].abs() + 64 * U32 * mag + TINY16, "dx")
    mag = (state["dy"].double() * h * inv).abs().sum(0)
    within(got["dw"], want["dw"], (case["rows"] + 4) * U32 * mag, "dweight")


def check_dispatch(case, state, got, want):
    for k in ("slots", "pairs", "offsets"):
        assert torch.equal(got[k].long(), want[k].long()), k
    assert torch.equal(got["rows"].double(), want["rows"])
    assert got["scales"] is None or torch.equal(got["scales"].double(), want["scales"])


def check_combine(case, state, got, want):
    mag = torch.zeros_like(want)
    for j in range(case["topk"]):
        v, has = operators._row_choice(state, j)
        mag += v.abs() * torch.where(has, state["weights"][:, j].double(), 0.0)[:, None]
    # decoded codes are rounded to fp32 too
    within(got, want, U16 * want.abs() + (case["topk"] + 2) * U32 * mag + TINY16, "rows")


def check_combine_grad(case, state, got, want):
    within(got["drows"], want["drows"], (U16 + 2 * U32) * want["drows"].abs() + TINY16, "drows")
    dy = state["dy"].double().abs()
    mag = torch.stack([(operators._row_choice(state, j)[0].abs() * dy).sum(1) for j in range(case["topk"])], 1)
    within(got["dweights"], want["dweights"], (case["hidden"] + 6) * U32 * mag, "dweights")


@pytest.mark.parametrize("case", CASES)
def test_case(case, monkeypatch):
    require_gpu()
    state = operators.prepare(case, 11)
    monkeypatch.setattr(operators, "own", True)
    got = operators.run(state)
    torch.cuda.synchronize()
    want = operators.exact(case, 11)
    check = {"norm": check_norm, "norm_grad": check_norm_grad, "dispatch": check_dispatch,
             "combine": check_combine, "combine_grad": check_combine_grad}[case["op"]]
    check(case, state, got, want)
