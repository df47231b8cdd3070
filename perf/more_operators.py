"""Cases of the operators on both ends of the wire: an MoE layer served from
weights in the codec's formats, its routing and the routing's gradient, and the
norm and clipping of gradients.

``run`` computes each operator in plain torch operations, or, where ``own`` is
true, with the framework's entry points; ``exact`` computes the same from the
operators' definitions in 64 bits.  Five kinds of case (``op``):

  route        softmax of the router's logits, the top experts of each token,
               and their weights
  route_grad   the gradient of the logits
  experts      a whole MoE layer for a few tokens: each token's experts
               (gate, up, down), weighted and summed
  grad_norm    the sum of squares over many gradient tensors
  grad_clip    gradients scaled in place to a largest norm, whose square's sum
               over all ranks is at hand
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "mx8": torch.float8_e4m3fn}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0, "mx8": 448.0}
GROUP = {"e4m3": 128, "e5m2": 128, "mx8": 32}
MAX_NORM = 1.0

# Most of a drawn case: logits, elements of all experts' matrices and of the
# pairs' ones, elements of all gradients (clipped ones: they are kept twice).
LOGITS = 16384 * 128
EXPERT_ELEMS = 8 * 3 * 4096 * 14336
PAIR_ELEMS = 256 * 3 * 4096 * 14336
NORM_ELEMS = 3_500_000_000
CLIP_ELEMS = 3 * 128 * 768 * 2048
TENSORS = 400


def listed():
    return [
        # One token being generated, its 8 of 128 experts.  Latency.
        dict(name="route token", op="route", tokens=1, topk=8, experts=128, dtype="f32", normalize=True,
             masked=0.0),
        # A training step's tokens.
        dict(name="route large", op="route", tokens=16384, topk=8, experts=128, dtype="f32", normalize=True,
             masked=0.0),
        # A packed batch: padding tokens have no expert, some experts are
        # switched off; weights are not renormalised.
        dict(name="route grad ragged", op="route_grad", tokens=777, topk=6, experts=60, dtype="bf16",
             normalize=False, masked=0.15),
        # A training step's tokens.
        dict(name="route grad large", op="route_grad", tokens=16384, topk=8, experts=128, dtype="f32",
             normalize=True, masked=0.0),
        # One token being generated, through the MoE layer that the benchmark
        # quantizes, in MXFP8.  Latency, and 38 MB of weights.
        dict(name="experts token", op="experts", tokens=1, topk=8, experts=128, hidden=2048, inter=768,
             fmt="mx8", dropped=0.0),
        # A batch of requests, a token each: most of the layer's experts.
        dict(name="experts batch", op="experts", tokens=32, topk=8, experts=128, hidden=2048, inter=768,
             fmt="mx8", dropped=0.0),
        # A ragged batch on one of several GPUs: padding tokens, experts that
        # live elsewhere, odd sizes, block-128 weights.
        dict(name="experts ragged", op="experts", tokens=13, topk=6, experts=60, hidden=1411, inter=1000,
             fmt="e4m3", dropped=0.15),
        # A large batch through few wide experts, in bf16.
        dict(name="experts large", op="experts", tokens=128, topk=2, experts=8, hidden=4096, inter=14336,
             fmt="bf16", dropped=0.0),
        # The small parameters of a layer (norms, biases).  Latency.
        dict(name="grad norm small", op="grad_norm", tensors=7, elems=9000, kind="f32"),
        # The whole gradient that the benchmark transfers, in bf16.
        dict(name="grad norm large", op="grad_norm", tensors=218, elems=NORM_ELEMS, kind="bf16"),
        # A shard of many odd tensors, views of flat buffers: fp32, bf16, and
        # 8-bit gradients, whose scales alone are written.
        dict(name="grad clip ragged", op="grad_clip", tensors=291, elems=40_000_001, kind="mixed"),
        # The gradient of the MoE layer that the benchmark quantizes, in fp32.
        dict(name="grad clip large", op="grad_clip", tensors=3, elems=CLIP_ELEMS, kind="f32"),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over [lo, hi] by its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def _size(rng, fmt, most):
    """A matrix's size: a multiple of 128, of 8, or odd (MXFP8: of 32)."""
    n = _spread(rng, 64, most)
    if fmt == "mx8":
        return n // 32 * 32
    kind = rng.random()
    if kind < 0.5:
        return max(128, n // 128 * 128)
    return n // 8 * 8 if kind < 0.8 else n | 1


def draw(rng):
    op = rng.choice(["route", "route_grad", "experts", "experts", "experts", "grad_norm", "grad_clip"])
    if op in ("route", "route_grad"):
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256, 512])
        return dict(op=op, tokens=_spread(rng, 1, LOGITS // experts), topk=rng.choice([1, 2, 4, 6, 8]),
                    experts=experts, dtype=rng.choice(["f32", "f32", "bf16"]),
                    normalize=rng.random() < 0.6, masked=rng.choice([0.0, 0.0, 0.15]))
    if op == "experts":
        fmt = rng.choice(["mx8", "mx8", "e4m3", "e5m2", "bf16"])
        experts = rng.choice([8, 16, 60, 64, 128, 160, 256])
        topk = rng.choice([1, 2, 4, 6, 8])
        hidden = _size(rng, fmt, 4096)
        inter = _size(rng, fmt, min(14336, EXPERT_ELEMS // (3 * experts * hidden)))
        tokens = _spread(rng, 1, min(128, PAIR_ELEMS // (3 * topk * hidden * inter)))
        return dict(op=op, tokens=tokens, topk=topk, experts=experts, hidden=hidden, inter=inter, fmt=fmt,
                    dropped=rng.choice([0.0, 0.0, 0.15]))
    tensors = _spread(rng, 1, TENSORS)
    kind = rng.choice(["f32", "bf16", "bf16", "e4m3", "mixed"])
    most = CLIP_ELEMS if op == "grad_clip" else NORM_ELEMS // 2 if kind == "f32" else NORM_ELEMS
    return dict(op=op, tensors=tensors, elems=_spread(rng, 8 * tensors, most), kind=kind)


def _tensors(case):
    """(kind, size) of each gradient of a list: a few large ones and many small
    ones, most of odd sizes."""
    rng = random.Random("%d %d %s" % (case["tensors"], case["elems"], case["kind"]))
    spread = 2.0 if case["tensors"] > 8 else 0.3 if case["tensors"] > 3 else 0.0
    shares = [math.exp(rng.gauss(0.0, spread)) for _ in range(case["tensors"])]
    whole = sum(shares)
    sizes = [max(1, int(case["elems"] * s / whole)) for s in shares]
    kinds = ["f32", "bf16", "bf16", "e4m3", "e5m2", "tensorwise"] if case["kind"] == "mixed" else [case["kind"]]
    return [(rng.choice(kinds), n) for n in sizes]


# --------------------------------------------------------------------------- #
# inputs                                                                      #
# --------------------------------------------------------------------------- #

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device=DEVICE, dtype=torch.float32)


def _logits(g, case):
    """A router's logits, some experts more popular than others; a share of the
    experts is switched off for a token, and as many tokens are padding."""
    tokens, experts = case["tokens"], case["experts"]
    l = _randn(g, experts) + _randn(g, tokens, experts) * 2.0
    if case["masked"] > 0.0:
        off = (_rand(g, tokens, experts) < case["masked"]) | (_rand(g, tokens, 1) < case["masked"])
        l = torch.where(off, -math.inf, l)
    return l if case["dtype"] == "f32" else l.to(torch.bfloat16)


def _matrices(g, fmt, experts, rows, width):
    """The experts' matrices [experts, rows, width] as a layer's initialisation
    leaves them, uniform, in their format: codes and scales, or bf16 and None."""
    parts, scales = [], []
    step = max(1, (1 << 27) // (rows * width))
    for e0 in range(0, experts, step):
        n = min(step, experts - e0)
        w = (_rand(g, n, rows, width) * 2.0 - 1.0) * (width ** -0.5)
        if fmt == "bf16":
            parts.append(w.to(torch.bfloat16))
            continue
        group = GROUP[fmt]
        blocks = -(-width // group)
        if blocks * group != width:
            w = torch.nn.functional.pad(w, (0, blocks * group - width))
        w = w.view(n, rows, blocks, group)
        amax = w.abs().amax(3)
        if fmt == "mx8":
            code = ((amax.view(torch.int32) >> 23) - 8).clamp(min=0)
            scales.append(code.to(torch.uint8))
            w = w * torch.exp2(127.0 - code.float())[..., None]
        else:
            s = (amax / FP8_MAX[fmt]).clamp(min=2.0 ** -126)
            scales.append(s)
            w = w / s[..., None]
        q = w.clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(FP8[fmt]).view(torch.uint8)
        parts.append(q.view(n, rows, blocks * group)[:, :, :width])
    return torch.cat(parts).contiguous(), torch.cat(scales) if scales else None


def _gradients(g, kind, sizes):
    """Gradients of the given sizes, views of one flat buffer as a trainer lays
    them out: the buffers that clipping writes (values, or codes' scales), the
    gradients, and their scales or None."""
    whole = sum(sizes)
    if kind in ("f32", "bf16"):
        v = torch.empty(whole, dtype=torch.float32 if kind == "f32" else torch.bfloat16, device=DEVICE)
        for a in range(0, whole, 1 << 27):
            v[a:a + (1 << 27)] = _randn(g, min(1 << 27, whole - a)) * 1e-3
        return v, list(v.split(sizes)), [None] * len(sizes)
    fmt = "e5m2" if kind == "e5m2" else "e4m3"
    q = torch.empty(whole, dtype=torch.uint8, device=DEVICE)
    for a in range(0, whole, 1 << 27):
        part = _randn(g, min(1 << 27, whole - a)) * (FP8_MAX[fmt] / 4)
        q[a:a + (1 << 27)] = part.clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(FP8[fmt]).view(torch.uint8)
    blocks = [1 if kind == "tensorwise" else -(-n // 128) for n in sizes]
    scales = torch.exp(_randn(g, sum(blocks))) * (4e-3 / FP8_MAX[fmt])
    return scales, list(q.split(sizes)), list(scales.split(blocks))


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("route", "route_grad"):
        s["logits"] = _logits(g, case)
        if case["op"] == "route_grad":
            s["weights"], s["ids"] = _plain_route(s)
            s["dweights"] = _randn(g, case["tokens"], case["topk"]) * 1e-2
    elif case["op"] == "experts":
        tokens, topk, experts, hidden, inter = (case[k] for k in ("tokens", "topk", "experts", "hidden", "inter"))
        s["x"] = _randn(g, tokens, hidden).to(torch.bfloat16)
        s["ids"] = torch.topk(_rand(g, tokens, experts), topk, dim=1).indices.to(torch.int32)
        s["weights"] = torch.softmax(_randn(g, tokens, topk), dim=1)
        if case["dropped"] > 0.0:
            gone = (_rand(g, tokens, 1) < case["dropped"]) | (_rand(g, tokens, topk) < case["dropped"])
            s["ids"] = torch.where(gone, -1, s["ids"])
        s["gate"], s["gate_scales"] = _matrices(g, case["fmt"], experts, inter, hidden)
        s["up"], s["up_scales"] = _matrices(g, case["fmt"], experts, inter, hidden)
        s["down"], s["down_scales"] = _matrices(g, case["fmt"], experts, hidden, inter)
    else:
        # a call is of one 8-bit format: E5M2 gradients are a list of their own
        s["lists"], s["written"] = {}, []
        tensors = _tensors(case)
        for kind in sorted({k for k, _ in tensors}):
            written, grads, scales = _gradients(g, kind, [n for k, n in tensors if k == kind])
            lists = s["lists"].setdefault("e5m2" if kind == "e5m2" else "e4m3", ([], []))
            lists[0].extend(grads)
            lists[1].extend(scales)
            s["written"].append(written)
        if case["op"] == "grad_clip":
            # over all ranks: a norm somewhat over the largest one
            norm = 1.01 + 0.04 * float(torch.rand((), generator=g, device=DEVICE))
            s["sumsq"] = torch.full((1,), (MAX_NORM * norm) ** 2, dtype=torch.float64, device=DEVICE)
    return s


# --------------------------------------------------------------------------- #
# one pass                                                                    #
# --------------------------------------------------------------------------- #

def _own(s):
    import dequantize_reduce_transfer_amd as fq

    fmts = {"e4m3": fq.E4M3, "e5m2": fq.E5M2}
    op = s["op"]
    if op == "route":
        weights, ids = fq.fp8q_moe_route(s["logits"], s["topk"], normalize=s["normalize"])
        return {"weights": weights, "ids": ids}
    if op == "route_grad":
        return fq.fp8q_moe_route_backward(s["dweights"], s["logits"], s["weights"], s["ids"],
                                          normalize=s["normalize"])
    if op == "experts":
        return fq.fp8q_moe_experts(s["x"], s["ids"], s["weights"], s["gate"], s["up"], s["down"],
                                   gate_scales=s["gate_scales"], up_scales=s["up_scales"],
                                   down_scales=s["down_scales"], fmt=fmts.get(s["fmt"], fq.E4M3))
    if op == "grad_norm":
        return [fq.fp8q_grad_sumsq(grads, scales=scales, fmt=fmts[fmt])
                for fmt, (grads, scales) in s["lists"].items()]
    norms = [fq.fp8q_grad_clip(grads, s["sumsq"], MAX_NORM, scales=scales, fmt=fmts[fmt])
             for fmt, (grads, scales) in s["lists"].items()]
    return {"norm": norms[0], "grads": s["written"]}


def _plain_route(s):
    l, topk = s["logits"].float(), s["topk"]
    order = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = order.values[:, :topk], order.indices[:, :topk]
    has = top != -math.inf
    most = torch.where(has[:, :1], order.values[:, :1], 0.0)
    e = torch.where(has, torch.exp(top - most), 0.0)
    whole = e.sum(1, keepdim=True) if s["normalize"] else torch.exp(l - most).sum(1, keepdim=True)
    return torch.where(has, e / whole, 0.0), torch.where(has, ids, -1).to(torch.int32)


def _plain_route_grad(s):
    l, w, dw = s["logits"].float(), s["weights"], s["dweights"]
    has = s["ids"] >= 0
    t = torch.where(has, w * dw, 0.0)
    total = t.sum(1, keepdim=True)
    if s["normalize"]:
        d = torch.zeros_like(l)
        t = torch.where(has, w * (dw - total), 0.0)
    else:
        most = l.amax(1, keepdim=True)
        e = torch.exp(l - torch.where(most != -math.inf, most, 0.0))
        d = -(e / e.sum(1, keepdim=True).clamp(min=1.0)) * total
    d = d.scatter_add(1, s["ids"].clamp(min=0).to(torch.int64), t)
    return d.to(s["logits"].dtype)


def _values(s, name, chosen):
    """The fp32 values of the chosen experts' matrices."""
    m, scales = s[name][chosen], s[name + "_scales"]
    if scales is None:
        return m.float()
    v = m.view(FP8[s["fmt"]]).float()
    scales = scales[chosen]
    if s["fmt"] == "mx8":
        scales = scales.view(torch.float8_e8m0fnu).float()
    return v * scales.repeat_interleave(GROUP[s["fmt"]], -1)[..., :v.shape[-1]]


def _plain_experts(s):
    x, held = s["x"].float(), (s["ids"] >= 0) & (s["ids"] < s["experts"])
    w = torch.where(held, s["weights"], 0.0)
    out = torch.zeros(x.shape, device=x.device)
    if s["ids"].numel() <= s["experts"]:
        # a choice at a time: each token's own matrices
        for j in range(s["topk"]):
            chosen = torch.where(held[:, j], s["ids"][:, j], 0).to(torch.int64)
            gate = torch.matmul(_values(s, "gate", chosen), x[:, :, None])
            up = torch.matmul(_values(s, "up", chosen), x[:, :, None])
            y = torch.matmul(_values(s, "down", chosen), gate / (1.0 + torch.exp(-gate)) * up)
            out = out + y[:, :, 0] * w[:, j:j + 1]
    else:
        # an expert at a time: all tokens through it, weighted by their choices
        for e in range(s["experts"]):
            gate = torch.matmul(x, _values(s, "gate", e).T)
            up = torch.matmul(x, _values(s, "up", e).T)
            y = torch.matmul(gate / (1.0 + torch.exp(-gate)) * up, _values(s, "down", e).T)
            out = out + y * torch.where(s["ids"] == e, w, 0.0).sum(1, keepdim=True)
    return out.to(torch.bfloat16)


def _decoded(v, scales, fmt):
    """A gradient's fp32 values."""
    if scales is None:
        return v.float()
    v = v.view(FP8[fmt]).float()
    return v * (scales if scales.numel() == 1 else scales.repeat_interleave(128)[:v.numel()])


def _plain_grad_norm(s):
    out = []
    for fmt, lists in s["lists"].items():
        total = torch.zeros(1, dtype=torch.float64, device=DEVICE)
        for v, scales in zip(*lists):
            for a in range(0, v.numel(), 1 << 28):
                part = v[a:a + (1 << 28)]
                blocks = scales
                if scales is not None and scales.numel() > 1:
                    blocks = scales[a // 128:(a + part.numel() + 127) // 128]
                total += _decoded(part, blocks, fmt).double().square().sum()
        out.append(total)
    return out


def _plain_grad_clip(s):
    norm = torch.sqrt(s["sumsq"])
    c = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0).float()
    for grads, scales in s["lists"].values():
        for v, q in zip(grads, scales):
            if q is not None:
                q.mul_(c)
            elif v.dtype == torch.float32:
                v.mul_(c)
            else:
                v.copy_(v.float() * c)
    return {"norm": norm.float(), "grads": s["written"]}


PLAIN = {"route": lambda s: dict(zip(("weights", "ids"), _plain_route(s))), "route_grad": _plain_route_grad,
         "experts": _plain_experts, "grad_norm": _plain_grad_norm, "grad_clip": _plain_grad_clip}


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------------------------------- #
# the same from the definitions, in 64 bits                                   #
# --------------------------------------------------------------------------- #

def _exact_route(s):
    """One choice after the other: the largest logit that is left, the lowest
    index where several are."""
    left = s["logits"].double()
    dead = left == -math.inf
    top = left.max(1, keepdim=True).values
    e = torch.exp(left - top).masked_fill(dead, 0.0)
    left, ids, parts = left.clone(), [], []
    for _ in range(s["topk"]):
        best = left.max(1, keepdim=True).values
        at = (left == best).to(torch.int8).argmax(1, keepdim=True)
        none = best == -math.inf
        ids.append(at.masked_fill(none, -1))
        parts.append(e.gather(1, at).masked_fill(none, 0.0))
        left.scatter_(1, at, -math.inf)
    ids, parts = torch.cat(ids, 1), torch.cat(parts, 1)
    whole = parts.sum(1, keepdim=True) if s["normalize"] else e.sum(1, keepdim=True)
    return {"weights": torch.where(ids >= 0, parts / whole, 0.0), "ids": ids}


def _exact_route_grad(s):
    """Through the matrix of the softmax's derivatives, a choice at a time."""
    l, ids = s["logits"].double(), s["ids"].long()
    held = ids >= 0
    w, dw = s["weights"].double(), s["dweights"].double().masked_fill(~held, 0.0)
    d = torch.zeros_like(l)
    if s["normalize"]:
        for i in range(s["topk"]):
            own_ = sum(w[:, j] * ((1.0 if i == j else 0.0) - w[:, i]) * dw[:, j] for j in range(s["topk"]))
            rows = held[:, i].nonzero()[:, 0]
            d[rows, ids[rows, i]] += own_[rows]
        return d
    live = held.any(1)
    p = torch.softmax(l[live], 1)
    dp = torch.zeros_like(p)
    for j in range(s["topk"]):
        rows = held[live, j].nonzero()[:, 0]
        dp[rows, ids[live][rows, j]] += dw[live][rows, j]
    d[live] = p * (dp - torch.einsum("te,te->t", p, dp)[:, None])
    return d


def _exact_matrix(s, name, e):
    m, scales = s[name][e], s[name + "_scales"]
    if scales is None:
        return m.double()
    column = torch.arange(m.shape[1], device=m.device) // GROUP[s["fmt"]]
    size = scales[e]
    if s["fmt"] == "mx8":
        size = torch.exp2(size.double() - 127.0)
    return m.view(FP8[s["fmt"]]).double() * size.double()[:, column]


def _exact_experts(s):
    """Expert by expert, the pairs that chose it."""
    x, ids = s["x"].double(), s["ids"].long()
    out = torch.zeros_like(x)
    for e in range(s["experts"]):
        token, choice = (ids == e).nonzero(as_tuple=True)
        if token.numel() == 0:
            continue
        rows = x[token]
        a = rows @ _exact_matrix(s, "gate", e).T
        h = a * torch.sigmoid(a) * (rows @ _exact_matrix(s, "up", e).T)
        y = h @ _exact_matrix(s, "down", e).T
        out.index_add_(0, token, y * s["weights"][token, choice].double()[:, None])
    return out


def _exact_grad_norm(s):
    out = []
    for fmt, (grads, scales) in s["lists"].items():
        total = torch.zeros(1, dtype=torch.float64, device=DEVICE)
        for v, q in zip(grads, scales):
            for a in range(0, v.numel(), 1 << 26):
                part = v[a:a + (1 << 26)]
                if q is not None:
                    at = torch.arange(a, a + part.numel(), device=v.device) // 128
                    size = q.expand(part.numel()) if q.numel() == 1 else q[at]
                    part = part.view(FP8[fmt]).float() * size      # values are fp32
                part = part.double()
                total += torch.dot(part, part)
        out.append(total)
    return out


def _exact_grad_clip(s):
    norm = s["sumsq"] ** 0.5
    share = torch.minimum(torch.ones_like(norm), MAX_NORM / (norm + 1e-6))
    return {"norm": norm, "grads": [v.double() * share for v in s["written"]]}


EXACT = {"route": _exact_route, "route_grad": _exact_route_grad, "experts": _exact_experts,
         "grad_norm": _exact_grad_norm, "grad_clip": _exact_grad_clip}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


# --------------------------------------------------------------------------- #
# what a pass cannot do without                                               #
# --------------------------------------------------------------------------- #

def work(case):
    op = case["op"]
    if op in ("route", "route_grad"):
        logits, pairs = case["tokens"] * case["experts"], case["tokens"] * case["topk"]
        size = 4 if case["dtype"] == "f32" else 2
        if op == "route":
            return {"bytes": logits * size + 8 * pairs, "flops": 4 * logits}
        if case["normalize"]:
            return {"bytes": logits * size + 12 * pairs, "flops": 4 * pairs}
        return {"bytes": 2 * logits * size + 12 * pairs, "flops": 6 * logits + 2 * pairs}
    if op == "experts":
        tokens, topk, experts, hidden, inter = (case[k] for k in ("tokens", "topk", "experts", "hidden", "inter"))
        # of the choices, those that neither their token nor they themselves
        # lose; and the experts that one of them names, on average
        kept = (1.0 - case["dropped"]) ** 2
        named = experts * (1.0 - (1.0 - kept * topk / experts) ** tokens)
        elems = hidden * inter
        if case["fmt"] == "bf16":
            matrices = 6 * elems
        elif case["fmt"] == "mx8":
            matrices = 3 * (elems + elems // 32)
        else:
            matrices = 3 * elems + 4 * (2 * inter * -(-hidden // 128) + hidden * -(-inter // 128))
        return {"bytes": named * matrices + tokens * (4 * hidden + 8 * topk),
                "flops": 6 * kept * tokens * topk * elems}
    size = {"f32": 4, "bf16": 2}
    total = 0
    for kind, n in _tensors(case):
        scales = 0 if kind in size else 4 if kind == "tensorwise" else 4 * -(-n // 128)
        if op == "grad_norm":
            total += n * size.get(kind, 1) + scales
        else:
            total += 2 * (n * size[kind] if kind in size else scales)
    elems = sum(n for _, n in _tensors(case))
    return {"bytes": total + 8, "flops": (2 if op == "grad_norm" else 1) * elems}
