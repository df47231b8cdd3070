"""Plain forms of the model's operators on the CPU, from their definitions in
64 bits, with the bounds that fp32 kernels of any summation order keep.  No
code is shared with the library."""
from __future__ import annotations

import numpy as np

from layer_ref import E4M3, E5M2, MX8, TINY16, U16, U32, decode_rows  # noqa: F401

BF16 = -1                              # a format beside layer_ref's
EXP = 3 * U32                          # an fp32 exp: within 1.5 ulps


def route(logits, topk, normalize):
    """(weights, ids, bound) in 64 bits; logits [tokens, experts] of values that
    are exact in fp32."""
    l = np.asarray(logits, np.float64)
    tokens, experts = l.shape
    ids = np.full((tokens, topk), -1, np.int64)
    w, bound = np.zeros((tokens, topk)), np.zeros((tokens, topk))
    for t in range(tokens):
        # NaN first, then the largest; equal ones (-0 and +0) by their index
        key = [(not np.isnan(l[t, i]), -l[t, i] if not np.isnan(l[t, i]) else 0.0, i) for i in range(experts)]
        order = [i for _, _, i in sorted(key) if not l[t, i] == -np.inf]
        chosen = order[:topk]
        ids[t, :len(chosen)] = chosen
        if not chosen:
            continue
        with np.errstate(all="ignore"):
            d = l[t] - l[t, order[0]]
            e = np.exp(d)
            e[l[t] == -np.inf] = 0.0
            over = chosen if normalize else order
            s = e[over].sum()
            w[t, :len(chosen)] = e[chosen] / s
            # d is rounded, exp is, and the sum's terms and additions are
            dist = np.where(e > 0, np.abs(d), 0.0)
            sum_err = (e[over] * (dist[over] * U32 + EXP)).sum() / s + (len(over) + 8) * U32
            bound[t, :len(chosen)] = w[t, :len(chosen)] * (np.abs(d[chosen]) * U32 + EXP + sum_err + 2 * U32) + 2.0 ** -140
    return w, ids, bound


def route_grad(dweights, logits, weights, ids, normalize):
    """(dlogits, bound) in 64 bits from the fp32 weights of the forward pass."""
    l = np.asarray(logits, np.float64)
    dw, w = np.asarray(dweights, np.float64), np.asarray(weights, np.float64)
    d, bound = np.zeros(l.shape), np.zeros(l.shape)
    for t in range(l.shape[0]):
        held = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < l.shape[1]]
        s = sum(w[t, j] * dw[t, j] for j in held)
        mag = sum(abs(w[t, j] * dw[t, j]) for j in held)
        for j in held:
            i = ids[t, j]
            term = w[t, j] * (dw[t, j] - s) if normalize else w[t, j] * dw[t, j]
            d[t, i] += term
            bound[t, i] += (4 + len(held)) * U32 * abs(w[t, j]) * (abs(dw[t, j]) + 4 * mag)
        live = l[t] != -np.inf
        if not normalize and live.any():
            with np.errstate(all="ignore"):
                dist = np.where(live, l[t] - l[t][live].max(), 0.0)
                e = np.where(live, np.exp(dist), 0.0)
                p = e / e.sum()
                d[t] -= p * s
                rel = np.abs(dist) * U32 + EXP + (e * (np.abs(dist) * U32 + EXP)).sum() / e.sum()
                bound[t] += p * mag * (rel + (l.shape[1] + 16) * U32) + U32 * np.abs(d[t])
    return d, bound + 2.0 ** -140


def silu(g):
    with np.errstate(all="ignore"):
        return g / (1.0 + np.exp(-g))


def experts(x, ids, weights, gate, up, down, bf16_out):
    """(out, bound) in 64 bits; gate, up [experts, inter, hidden] and down
    [experts, hidden, inter] as values.

    The bound: a sum of n products in fp32, in any order, is off by at most
    (n + 8) * U32 of the products' magnitudes; silu has a slope of at most 1.1
    and five roundings; for bf16 output h is held to 2^-15 of itself (its eight
    leading bits and eight of the rest), else exactly, as 2 or 3 numbers whose
    products are summed together."""
    x = np.asarray(x, np.float64)
    out, bound = np.zeros(x.shape), np.zeros(x.shape)
    hidden, inter = x.shape[1], gate.shape[1]
    for t in range(ids.shape[0]):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < gate.shape[0]:
                continue
            w = float(weights[t, j])
            g, u = gate[e] @ x[t], up[e] @ x[t]
            eg = (hidden + 8) * U32 * (np.abs(gate[e]) @ np.abs(x[t]))
            eu = (hidden + 8) * U32 * (np.abs(up[e]) @ np.abs(x[t]))
            h = silu(g) * u
            eh = 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + (6 * U32 + EXP) * np.abs(h)
            if bf16_out:
                eh = eh + 2.0 ** -15 * np.abs(h)
            y = down[e] @ h
            ey = np.abs(down[e]) @ eh + (3 * inter + 24) * U32 * (np.abs(down[e]) @ (np.abs(h) + eh))
            out[t] += w * y
            bound[t] += abs(w) * (ey + (ids.shape[1] + 2) * U32 * np.abs(y))
    if bf16_out:
        bound += U16 * (np.abs(out) + bound) + TINY16
    return out, bound + 2.0 ** -140


def sumsq(values):
    """Sum of squares of a list of fp32 arrays, exactly rounded."""
    import math
    return math.fsum(float(v) * float(v) for a in values for v in np.asarray(a, np.float64).ravel())
