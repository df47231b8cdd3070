"""Cases of the MoE layer's activation operators: the residual stream's norm
into 8 bits and its gradient, and the rows' way to their experts and back.

``run`` computes each operator in plain torch operations, or, where ``own`` is
true, with the framework's entry points; ``exact`` computes the same from the
operators' definitions in 64 bits.  Five kinds of case (``op``):

  norm           h = x + residual, y = rms_norm(h) * weight, y in 8 bits with
                 scales (fp32 per 128 of a row, or E8M0 per 32), y in bf16
                 where a router needs it, 1/rms where a backward pass does
  norm_grad      the gradients of h (with the residual stream's own added)
                 and of the weight
  dispatch       the (token, choice) pairs sorted by expert, and the tokens'
                 rows written in that order
  combine        each token's expert rows, weighted and summed
  combine_grad   the gradients of the expert rows and of the weights
"""
import math

import torch
import torch.nn.functional as F

own = False

DEVICE = "cuda"
EPS = 1e-6
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "mx8": torch.float8_e4m3fn}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0, "mx8": 448.0}
GROUP = {"e4m3": 128, "e5m2": 128, "mx8": 32}

# Most elements (rows x hidden) of a drawn norm, and (pairs x hidden) of a
# drawn dispatch, combine or gradient: those of the largest listed ones.
NORM_ELEMS = 16384 * 8192
MOE_ELEMS = 16384 * 8 * 2048


def listed():
    return [
        # One token being generated: its row of the residual stream, on its
        # way into the experts.  Latency.
        dict(name="norm token", op="norm", rows=1, hidden=2048, fmt="e4m3", residual=True, y=False,
             rstd=False, weight="bf16"),
        # A batch of requests, a token each; the router reads the bf16 copy.
        dict(name="norm batch", op="norm", rows=96, hidden=4096, fmt="mx8", residual=True, y=True,
             rstd=False, weight="bf16"),
        # Ragged: an odd count of rows whose last block is partial, no
        # residual (a layer's first norm), fp32 weight, kept for a backward.
        dict(name="norm ragged", op="norm", rows=1021, hidden=1000, fmt="e5m2", residual=False, y=True,
             rstd=True, weight="f32"),
        # A long prompt, or a training step's tokens, at a large hidden size.
        dict(name="norm large", op="norm", rows=16384, hidden=8192, fmt="e4m3", residual=True, y=False,
             rstd=True, weight="bf16"),
        # A short packed batch in training, at a hidden size that is no
        # multiple of 128.
        dict(name="norm grad ragged", op="norm_grad", rows=509, hidden=2888, residual=True, weight="f32"),
        # A training step's tokens.
        dict(name="norm grad large", op="norm_grad", rows=16384, hidden=4096, residual=True, weight="bf16"),
        # One token to its 8 of 128 experts, MXFP8 rows.  Latency.
        dict(name="dispatch token", op="dispatch", tokens=1, topk=8, experts=128, hidden=2048, fmt="mx8",
             dropped=0.0),
        # A training step's tokens to the experts of the MoE layer.
        dict(name="dispatch large", op="dispatch", tokens=16384, topk=8, experts=128, hidden=2048,
             fmt="e4m3", dropped=0.0),
        # A few requests' tokens back from the experts, 8-bit rows.  Latency.
        dict(name="combine batch", op="combine", tokens=5, topk=8, experts=128, hidden=2048, fmt="e4m3",
             dropped=0.0),
        # A training step's tokens back from the experts.
        dict(name="combine large", op="combine", tokens=16384, topk=8, experts=128, hidden=2048, fmt="bf16",
             dropped=0.0),
        # A packed batch with padding tokens (no expert) and an odd hidden size.
        dict(name="combine grad ragged", op="combine_grad", tokens=777, topk=6, experts=60, hidden=1411,
             dropped=0.15),
        # A training step's gradient through the weighted sum.
        dict(name="combine grad large", op="combine_grad", tokens=16384, topk=8, experts=128, hidden=2048,
             dropped=0.0),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _apart(n, step=1):
    """n, moved by a step off a size that is left out everywhere."""
    return n + step if n == 3072 else n


def _hidden(rng, fmt, most):
    h = _spread(rng, 64, most)
    if fmt == "mx8":
        return _apart(max(64, h // 32 * 32), 32)
    kind = rng.random()
    if kind < 0.5:
        return _apart(max(128, h // 128 * 128), 128)
    if kind < 0.8:
        return _apart(max(64, h // 8 * 8), 8)
    return h | 1


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "dispatch", "combine", "combine_grad"])
    if op in ("norm", "norm_grad"):
        fmt = rng.choice(["e4m3", "e5m2", "mx8"]) if op == "norm" else "e4m3"
        hidden = _hidden(rng, fmt, 8192)
        most = NORM_ELEMS if op == "norm" else 16384 * 4096
        rows = _apart(_spread(rng, 1, min(16384, most // hidden)))
        case = dict(op=op, rows=rows, hidden=hidden, residual=rng.random() < 0.75,
                    weight=rng.choice(["bf16", "f32"]))
        if op == "norm":
            case.update(fmt=fmt, y=rng.random() < 0.5, rstd=rng.random() < 0.5)
        return case
    fmt = {"dispatch": rng.choice(["e4m3", "mx8", "bf16"]),
           "combine": rng.choice(["e4m3", "e5m2", "mx8", "bf16", "bf16"]), "combine_grad": "bf16"}[op]
    topk = rng.choice([1, 2, 4, 6, 8])
    hidden = _hidden(rng, fmt, 4096)
    tokens = _spread(rng, 1, min(16384, MOE_ELEMS // (topk * hidden)))
    while 3072 in (tokens, tokens * topk):
        tokens += 1
    case = dict(op=op, tokens=tokens, topk=topk, experts=rng.choice([8, 16, 60, 64, 128, 160, 256]),
                hidden=hidden, dropped=rng.choice([0.0, 0.0, 0.1, 0.5]))
    if op != "combine_grad":
        case["fmt"] = fmt
    return case


# --------------------------------------------------------------------------- #
# inputs                                                                      #
# --------------------------------------------------------------------------- #

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _bf16(t):
    return t.to(torch.bfloat16)


def _stream_rows(g, rows, hidden):
    """Rows of a residual stream: each row at its own size, and one channel
    in a hundred or so far larger than the rest."""
    channel = torch.where(_rand(g, hidden) < 0.01, 20.0, 1.0)
    return _randn(g, rows, hidden) * channel * torch.exp(_randn(g, rows, 1) * 0.5)


def _codes(g, rows, hidden, fmt):
    """8-bit rows with their scales, as a quantize leaves them: the largest
    code of a block near the format's maximum, scales over a few decades."""
    blocks = -(-hidden // GROUP[fmt])
    top = FP8_MAX[fmt]
    q = (_randn(g, rows, hidden) * (top / 4)).clamp(-top, top).to(FP8[fmt]).view(torch.uint8)
    if fmt == "mx8":
        return q, torch.randint(110, 122, (rows, blocks), generator=g, device=DEVICE, dtype=torch.uint8)
    return q, torch.exp(_randn(g, rows, blocks)) * (1.0 / top)


def _choices(g, case):
    """Each token's experts, distinct, some experts more popular than others;
    a share of the tokens (padding) has none, and as many single choices are
    left out too (experts that live elsewhere).  Returns ids and weights."""
    tokens, topk, experts = case["tokens"], case["topk"], case["experts"]
    liking = _randn(g, experts) + _randn(g, tokens, experts) * 2.0
    score, ids = torch.topk(liking, topk, dim=1)
    weights = torch.softmax(score, dim=1)
    ids = ids.to(torch.int32)
    if case["dropped"] > 0.0:
        gone = (_rand(g, tokens, 1) < case["dropped"]) | (_rand(g, tokens, topk) < case["dropped"])
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids.contiguous(), weights.contiguous()


def _places(ids, experts):
    """Where each pair goes (-1: nowhere), which pair is at each place, and
    each expert's first place, by a stable sort."""
    flat = ids.reshape(-1).to(torch.int64)
    pairs = flat.numel()
    held = (flat >= 0) & (flat < experts)
    key = torch.where(held, flat, experts)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(pairs, device=flat.device)
    slots = torch.where(held, place, -1)
    count = held.sum()
    at = torch.where(torch.arange(pairs, device=flat.device) < count, order, -1)
    sizes = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device)
    sizes.index_add_(0, key, torch.ones_like(key))
    offsets = torch.cumsum(sizes, 0) - sizes
    return slots.reshape(ids.shape).to(torch.int32), at.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("norm", "norm_grad"):
        rows, hidden = case["rows"], case["hidden"]
        weight = 1.0 + 0.2 * _randn(g, hidden)
        s["w"] = _bf16(weight) if case["weight"] == "bf16" else weight
    if case["op"] == "norm":
        s["x"] = _bf16(_randn(g, rows, hidden) if case["residual"] else _stream_rows(g, rows, hidden))
        s["res"] = _bf16(_stream_rows(g, rows, hidden)) if case["residual"] else None
    elif case["op"] == "norm_grad":
        s["h"] = _bf16(_stream_rows(g, rows, hidden))
        s["inv"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
        s["dy"] = _bf16(_randn(g, rows, hidden) * 1e-2)
        s["dh"] = _bf16(_randn(g, rows, hidden) * 1e-2) if case["residual"] else None
    else:
        tokens, hidden = case["tokens"], case["hidden"]
        pairs = tokens * case["topk"]
        s["ids"], s["weights"] = _choices(g, case)
        if case["op"] == "dispatch":
            if case["fmt"] == "bf16":
                s["x"], s["scales"] = _bf16(_randn(g, tokens, hidden)), None
            else:
                s["x"], s["scales"] = _codes(g, tokens, hidden, case["fmt"])
            # The receive buffers, which the program keeps; places past the
            # last pair stay as they are.
            s["rows"] = torch.zeros(pairs, hidden, dtype=s["x"].dtype, device=DEVICE)
            s["rows_scales"] = None if s["scales"] is None else torch.zeros(
                pairs, s["scales"].shape[1], dtype=s["scales"].dtype, device=DEVICE)
        else:
            s["slots"] = _places(s["ids"], case["experts"])[0]
            if case["op"] == "combine" and case["fmt"] != "bf16":
                s["rows"], s["scales"] = _codes(g, pairs, hidden, case["fmt"])
            else:
                s["rows"], s["scales"] = _bf16(_randn(g, pairs, hidden)), None
            if case["op"] == "combine_grad":
                s["dy"] = _bf16(_randn(g, tokens, hidden) * 1e-2)
                s["drows"] = torch.zeros(pairs, hidden, dtype=torch.bfloat16, device=DEVICE)
    return s


# --------------------------------------------------------------------------- #
# one pass                                                                    #
# --------------------------------------------------------------------------- #

def _as_fp8(q, fmt):
    return q.view(FP8[fmt])


def _as_scales(s, fmt):
    return s.view(torch.float8_e8m0fnu) if fmt == "mx8" else s


def _own(s):
    import dequantize_reduce_transfer_amd as fq

    fmts = {"e4m3": fq.E4M3, "e5m2": fq.E5M2}
    op = s["op"]
    if op == "norm":
        if s["fmt"] == "mx8":
            out = fq.mx8_rms_norm_quantize(s["x"], s["w"], EPS, residual=s["res"], want_y=s["y"],
                                           want_rstd=s["rstd"])
        else:
            out = fq.fp8q_rms_norm_quantize(s["x"], s["w"], EPS, residual=s["res"], fmt=fmts[s["fmt"]],
                                            want_y=s["y"], want_rstd=s["rstd"])
        return {"q": _as_fp8(out.q, s["fmt"]), "scales": _as_scales(out.scales, s["fmt"]),
                "h": out.h if s["residual"] else None, "y": out.y, "rstd": out.rstd}
    if op == "norm_grad":
        dx, dw = fq.fp8q_rms_norm_backward(s["dy"], s["h"], s["w"], s["inv"], dh=s["dh"])
        return {"dx": dx, "dw": dw}
    if op == "dispatch":
        slots, pairs, offsets = fq.fp8q_moe_sort(s["ids"], s["experts"])
        rows, scales = fq.fp8q_moe_permute(s["x"], slots, scales=s["scales"], out=s["rows"],
                                           scales_out=s["rows_scales"])
        return {"slots": slots, "pairs": pairs, "offsets": offsets,
                "rows": rows if s["fmt"] == "bf16" else _as_fp8(rows, s["fmt"]),
                "scales": None if scales is None else _as_scales(scales, s["fmt"])}
    if op == "combine":
        return fq.fp8q_moe_combine(s["rows"], s["slots"], s["weights"], scales=s["scales"],
                                   fmt=fmts.get(s["fmt"], fq.E4M3))
    drows, dw = fq.fp8q_moe_combine_backward(s["dy"], s["rows"], s["slots"], s["weights"],
                                             drows_out=s["drows"])
    return {"drows": drows, "dweights": dw}


def _blocks(y, group):
    """y's rows in blocks, the last one of a row filled up with zeros."""
    rows, hidden = y.shape
    blocks = -(-hidden // group)
    if blocks * group != hidden:
        y = F.pad(y, (0, blocks * group - hidden))
    return y.view(rows, blocks, group)


def _plain_norm(s):
    fmt, hidden = s["fmt"], s["hidden"]
    h = s["x"].float()
    if s["residual"]:
        h = h + s["res"].float()
    inv = torch.rsqrt(h.square().mean(1) + EPS)
    y = h * inv[:, None] * s["w"].float()
    b = _blocks(y, GROUP[fmt])
    amax = b.abs().amax(2)
    if fmt == "mx8":
        exponent = amax.view(torch.int32) >> 23            # amax >= 0: the biased exponent
        code = (exponent - 8).clamp(min=0)
        scales = code.to(torch.uint8)
        ratio = b * torch.exp2(127.0 - code.float())[:, :, None]
    else:
        scales = (amax / FP8_MAX[fmt]).clamp(min=2.0 ** -126)
        ratio = b / scales[:, :, None]
    q = ratio.clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(FP8[fmt]).view(y.shape[0], -1)
    if q.shape[1] != hidden:
        q = q.view(torch.uint8)[:, :hidden].contiguous().view(FP8[fmt])
    return {"q": q, "scales": _as_scales(scales, fmt), "h": _bf16(h) if s["residual"] else None,
            "y": _bf16(y) if s["y"] else None, "rstd": inv if s["rstd"] else None}


def _plain_norm_grad(s):
    h, g, inv = s["h"].float(), s["dy"].float() * s["w"].float(), s["inv"][:, None]
    c = (g * h).sum(1, keepdim=True) * inv * inv * inv / s["hidden"]
    dx = g * inv - h * c
    if s["residual"]:
        dx = dx + s["dh"].float()
    return {"dx": _bf16(dx), "dw": (s["dy"].float() * h * inv).sum(0)}


def _plain_dispatch(s):
    slots, pairs, offsets = _places(s["ids"], s["experts"])
    held = pairs >= 0
    token = torch.where(held, pairs, 0).to(torch.int64) // s["topk"]
    rows = torch.where(held[:, None], s["x"][token], 0).to(s["x"].dtype)
    scales = s["scales"]
    if scales is not None:
        scales = _as_scales(torch.where(held[:, None], scales[token], 0).to(scales.dtype), s["fmt"])
    return {"slots": slots, "pairs": pairs, "offsets": offsets,
            "rows": rows if s["fmt"] == "bf16" else _as_fp8(rows, s["fmt"]), "scales": scales}


def _values(s):
    """The expert rows as fp32 values."""
    if s["scales"] is None:
        return s["rows"].float()
    v = _as_fp8(s["rows"], s["fmt"]).float()
    scales = _as_scales(s["scales"], s["fmt"]).float()
    return v * scales.repeat_interleave(GROUP[s["fmt"]], 1)[:, :s["hidden"]]


def _plain_combine(s):
    held = s["slots"] >= 0
    at = torch.where(held, s["slots"], 0).to(torch.int64)
    w = torch.where(held, s["weights"], 0.0)
    picked = torch.where(held[:, :, None], _values(s)[at], 0.0)
    return _bf16((picked * w[:, :, None]).sum(1))


def _plain_combine_grad(s):
    held = s["slots"] >= 0
    at = torch.where(held, s["slots"], 0).to(torch.int64)
    dy = s["dy"].float()
    dw = (s["rows"].float()[at] * dy[:, None, :]).sum(2)
    drows = torch.zeros_like(s["drows"])
    drows[s["slots"][held].to(torch.int64)] = _bf16(s["weights"][:, :, None] * dy[:, None, :])[held]
    return {"drows": drows, "dweights": torch.where(held, dw, 0.0)}


PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "dispatch": _plain_dispatch,
         "combine": _plain_combine, "combine_grad": _plain_combine_grad}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------------------------------- #
# the same from the definitions, in 64 bits                                   #
# --------------------------------------------------------------------------- #

def _exact_norm(s):
    """q is the value that a code rounds: y over its block's scale."""
    fmt, rows, hidden = s["fmt"], s["rows"], s["hidden"]
    h = s["x"].double()
    if s["residual"]:
        h += s["res"].double()
    inv = (torch.einsum("rh,rh->r", h, h) / hidden + EPS) ** -0.5
    y = torch.einsum("rh,r,h->rh", h, inv, s["w"].double())
    group = GROUP[fmt]
    full = hidden // group * group
    amax = y[:, :full].abs().reshape(rows, full // group, group).max(2).values if full else y[:, :0]
    if full < hidden:
        amax = torch.cat([amax, y[:, full:].abs().max(1, keepdim=True).values], 1)
    if fmt == "mx8":
        scales = torch.exp2((torch.frexp(amax).exponent.double() - 1 - 8).clamp(-127, 127))
    else:
        scales = torch.maximum(amax / FP8_MAX[fmt], torch.full_like(amax, 2.0 ** -126))
    column = torch.arange(hidden, device=y.device) // group
    q = torch.clamp(y / scales[:, column], -FP8_MAX[fmt], FP8_MAX[fmt])
    return {"q": q, "scales": scales, "h": h if s["residual"] else None, "y": y if s["y"] else None,
            "rstd": inv if s["rstd"] else None}


def _exact_norm_grad(s):
    h, dy, inv = s["h"].double(), s["dy"].double(), s["inv"].double()
    unit = h * inv[:, None]                                 # the normed rows
    g = dy * s["w"].double()
    along = (unit * g).mean(1, keepdim=True)
    dx = inv[:, None] * (g - unit * along)
    if s["residual"]:
        dx += s["dh"].double()
    return {"dx": dx, "dw": torch.einsum("rh,rh->h", dy, unit)}


def _exact_dispatch(s):
    """The pairs of each expert, in order, from counts of what comes before."""
    ids = s["ids"].reshape(-1).long()
    experts, topk = s["experts"], s["topk"]
    at = torch.cat([(ids == e).nonzero()[:, 0] for e in range(experts)])
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = torch.stack([(ids == e).sum() for e in range(experts)]).cumsum(0)
    slots = torch.full_like(ids, -1)
    slots[at] = torch.arange(at.numel(), device=ids.device)
    pairs = torch.full_like(ids, -1)
    pairs[:at.numel()] = at
    values = s["x"].double() if s["fmt"] == "bf16" else _as_fp8(s["x"], s["fmt"]).double()
    rows = torch.zeros(ids.numel(), s["hidden"], dtype=torch.float64, device=ids.device)
    rows[:at.numel()] = values[at // topk]
    scales = None
    if s["scales"] is not None:
        sizes = _as_scales(s["scales"], s["fmt"]).double()
        # a place without a pair keeps its zero byte: 2^-127 as an E8M0 scale
        nothing = 2.0 ** -127 if s["fmt"] == "mx8" else 0.0
        scales = torch.full((ids.numel(), sizes.shape[1]), nothing, dtype=torch.float64, device=ids.device)
        scales[:at.numel()] = sizes[at // topk]
    return {"slots": slots.reshape(s["ids"].shape), "pairs": pairs, "offsets": offsets, "rows": rows,
            "scales": scales}


def _row_choice(s, j):
    """The j-th expert row of every token in 64 bits, zeros where it has none,
    and whether it has one."""
    slot = s["slots"][:, j].long()
    has = slot >= 0
    slot = slot.clamp(min=0)
    if s["scales"] is None:
        v = s["rows"][slot].double()
    else:
        column = torch.arange(s["hidden"], device=slot.device) // GROUP[s["fmt"]]
        v = _as_fp8(s["rows"][slot], s["fmt"]).double()
        v *= _as_scales(s["scales"][slot][:, column].contiguous(), s["fmt"]).double()
    return v.masked_fill_(~has[:, None], 0.0), has


def _exact_combine(s):
    out = torch.zeros(s["tokens"], s["hidden"], dtype=torch.float64, device=s["rows"].device)
    for j in range(s["topk"]):
        v, has = _row_choice(s, j)
        out += v * torch.where(has, s["weights"][:, j].double(), 0.0)[:, None]
    return out


def _exact_combine_grad(s):
    dy = s["dy"].double()
    drows = torch.zeros(s["rows"].shape, dtype=torch.float64, device=dy.device)
    dw = torch.zeros(s["tokens"], s["topk"], dtype=torch.float64, device=dy.device)
    for j in range(s["topk"]):
        v, has = _row_choice(s, j)
        dw[:, j] = torch.einsum("th,th->t", v, dy)
        drows[s["slots"][has, j].long()] = dy[has] * s["weights"][has, j].double()[:, None]
    return {"drows": drows, "dweights": dw}


EXACT = {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "dispatch": _exact_dispatch,
         "combine": _exact_combine, "combine_grad": _exact_combine_grad}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


# --------------------------------------------------------------------------- #
# what a pass cannot do without                                               #
# --------------------------------------------------------------------------- #

def _row_bytes(fmt, hidden):
    if fmt == "bf16":
        return 2 * hidden
    return hidden + (hidden // 32 if fmt == "mx8" else 4 * (-(-hidden // 128)))


def work(case):
    op, hidden = case["op"], case["hidden"]
    if op in ("norm", "norm_grad"):
        rows = case["rows"]
        bytes_ = hidden * (2 if case["weight"] == "bf16" else 4)
        if op == "norm":
            bytes_ += rows * (2 * hidden + _row_bytes(case["fmt"], hidden))
            bytes_ += rows * hidden * (4 if case["residual"] else 0) + rows * hidden * (2 if case["y"] else 0)
            bytes_ += 4 * rows if case["rstd"] else 0
            return {"bytes": bytes_, "flops": rows * hidden * (9 + (1 if case["residual"] else 0))}
        bytes_ += rows * hidden * (8 if case["residual"] else 6) + 4 * rows + 4 * hidden
        return {"bytes": bytes_, "flops": rows * hidden * 9}
    tokens = case["tokens"]
    pairs = tokens * case["topk"]
    # of the choices, those that neither their token nor they themselves lose
    held = pairs * (1.0 - case["dropped"]) ** 2
    if op == "dispatch":
        row = _row_bytes(case["fmt"], hidden)
        return {"bytes": 4 * pairs + 8 * pairs + 4 * (case["experts"] + 1) + tokens * row + held * row,
                "flops": 0}
    if op == "combine":
        row = _row_bytes(case["fmt"], hidden)
        return {"bytes": 8 * pairs + held * row + 2 * tokens * hidden, "flops": 2 * held * hidden}
    return {"bytes": 8 * pairs + 2 * tokens * hidden + 4 * held * hidden + 4 * pairs,
            "flops": 3 * held * hidden}
