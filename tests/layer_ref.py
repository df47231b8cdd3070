"""Plain forms of the layer operators on the CPU, from their definitions: in
64 bits (rms_norm, its gradients, the sort, combine and its gradients), and
the encode of fp32 rows step by step in fp32 with IEEE divides and the
oracle's converter, which the kernels' codes and scales must equal bit for
bit.  No code is shared with the library."""
from __future__ import annotations

import numpy as np

import oracle

U32 = 2.0 ** -24                       # rounding to fp32: at most U32 of the value
U16 = 2.0 ** -8                        # rounding to bf16 (8 significant bits)
TINY16 = 2.0 ** -126 * 2.0 ** -8       # and half a subnormal step below the normal range

E4M3, E5M2, MX8 = 0, 1, 2
FP8_MAX = {E4M3: 448.0, E5M2: 57344.0, MX8: 448.0}


def rms_norm(x, res, w, eps):
    """(h, rstd, y) in 64 bits."""
    h = np.asarray(x, np.float64)
    if res is not None:
        h = h + np.asarray(res, np.float64)
    rstd = 1.0 / np.sqrt((h * h).sum(1) / h.shape[1] + eps)
    return h, rstd, h * rstd[:, None] * np.asarray(w, np.float64)


def rms_norm_grads(dy, h, w, rstd, dh):
    """(dx, dw) in 64 bits, with rstd taken as a function of h."""
    dy, h, w = (np.asarray(t, np.float64) for t in (dy, h, w))
    rstd = np.asarray(rstd, np.float64)[:, None]
    g = dy * w
    c = rstd ** 3 * (g * h).sum(1, keepdims=True) / h.shape[1]
    dx = g * rstd - h * c
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * h * rstd).sum(0)


def norm_f32(x, res, w, rstd):
    """(h, y) in fp32, each step rounded as the operator defines it, from the
    fp32 rstd the device found."""
    h = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if res is not None:
            h = h + np.asarray(res, np.float32)
        y = (h * np.asarray(rstd, np.float32)[:, None]) * np.asarray(w, np.float32)
    return h, y


def encode_rows(y, fmt):
    """fp32 rows -> (codes [rows, hidden], scales [rows, blocks]) by the codec's
    rules: fp32 scales per 128 (the last block of a row partial), or E8M0 per 32."""
    y = np.asarray(y, np.float32)
    rows, hidden = y.shape
    block = 32 if fmt == MX8 else 128
    blocks = -(-hidden // block)
    codes = np.zeros((rows, hidden), np.uint8)
    scales = np.zeros((rows, blocks), np.uint8 if fmt == MX8 else np.float32)
    for b in range(blocks):
        part = y[:, b * block:(b + 1) * block]
        finite = np.isfinite(part).all(1)
        with np.errstate(all="ignore"):
            amax = np.where(finite, np.abs(part).max(1), np.float32(0)).astype(np.float32)
            if fmt == MX8:
                mant, ex = np.frexp(amax.astype(np.float64))
                X = np.where(amax > 0, np.clip(ex - 1 - 8, -127, 127), -127)
                ratio = np.ldexp(part.astype(np.float64), -X[:, None]).astype(np.float32)
                scales[:, b] = np.where(finite, X + 127, 255).astype(np.uint8)
                q = oracle.fp8_encode(np.where(finite[:, None], ratio, np.float32(0)), 0)
            else:
                s = np.maximum(amax / np.float32(FP8_MAX[fmt]), np.float32(2.0 ** -126)).astype(np.float32)
                ratio = (part / s[:, None]).astype(np.float32)
                scales[:, b] = np.where(finite, s, np.float32(np.nan))
                q = oracle.fp8_encode(np.where(finite[:, None], ratio, np.float32(0)), fmt)
        codes[:, b * block:(b + 1) * block] = np.where(finite[:, None], q, 0x7F)
    return codes, scales


def decode_rows(codes, scales, fmt):
    """The fp32 values of 8-bit rows (code * scale rounded to fp32)."""
    block = 32 if fmt == MX8 else 128
    v = oracle.fp8_decode(codes, 0 if fmt == MX8 else fmt)
    if fmt == MX8:
        s = np.ldexp(1.0, np.asarray(scales, np.int64) - 127)
        s[np.asarray(scales) == 255] = np.nan
    else:
        s = np.asarray(scales, np.float64)
    column = np.arange(codes.shape[1]) // block
    with np.errstate(all="ignore"):
        return (v.astype(np.float64) * s[:, column]).astype(np.float32)


def moe_sort(ids, experts):
    """(slots, pairs, offsets) by numpy's stable sort."""
    flat = np.asarray(ids).reshape(-1)
    held = (flat >= 0) & (flat < experts)
    at = np.nonzero(held)[0]
    order = at[np.argsort(flat[at], kind="stable")]
    slots = np.full(flat.size, -1, np.int32)
    slots[order] = np.arange(order.size)
    pairs = np.full(flat.size, -1, np.int32)
    pairs[:order.size] = order
    counts = np.bincount(flat[at].astype(np.int64), minlength=experts)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return slots.reshape(np.asarray(ids).shape), pairs, offsets


def combine(values, slots, weights):
    """(sum, sum of magnitudes) in 64 bits; values [n, hidden] fp32."""
    tokens, topk = slots.shape
    out = np.zeros((tokens, values.shape[1]))
    mag = np.zeros_like(out)
    for j in range(topk):
        has = (slots[:, j] >= 0) & (slots[:, j] < values.shape[0])
        v = values[np.where(has, slots[:, j], 0)].astype(np.float64) if values.shape[0] else 0.0 * out
        w = np.ones(tokens) if weights is None else weights[:, j].astype(np.float64)
        with np.errstate(all="ignore"):
            term = np.where(has[:, None], v * w[:, None], 0.0)
        out += term
        mag += np.abs(term)
    return out, mag


def combine_grads(dy, values, slots, weights):
    """(drows, dweights, sum of dweights' magnitudes) in 64 bits; rows that no
    slot names are NaN."""
    tokens, topk = slots.shape
    dy = np.asarray(dy, np.float64)
    drows = np.full(values.shape, np.nan)
    dw, mag = np.zeros((tokens, topk)), np.zeros((tokens, topk))
    for t in range(tokens):
        for j in range(topk):
            s = slots[t, j]
            if 0 <= s < values.shape[0]:
                drows[s] = dy[t] * float(weights[t, j])
                prod = dy[t] * values[s].astype(np.float64)
                dw[t, j], mag[t, j] = prod.sum(), np.abs(prod).sum()
    return drows, dw, mag


def differences(f, x, step):
    """Central differences of the scalar f at x, element by element."""
    x = np.array(x, np.float64)
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f(x)
        x[i] = keep - step
        down = f(x)
        x[i] = keep
        g[i] = (up - down) / (2 * step)
    return g
