"""The norm entry points against the plain forms of layer_ref.

What the device's rstd rounds to depends on the order of its sum, so it is
held to a derived bound against 64 bits; given that rstd, every other output
(codes, scales, h, y) is a fixed sequence of fp32 roundings and must be equal
bit for bit.

The bound on rstd.  The sum's terms are squares, so its relative error is at
most its longest chain of roundings times 2^-24: 8 V <= 32 in a lane, 6 across
the wave, 16 across the waves.  The rounding of h enters squared (2), dividing
by hidden and adding eps are 2 more: 58.  The square root halves that and adds
one rounding, the reciprocal another: 31, taken as 32.
"""
import numpy as np
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
import layer_ref as ref
from gpu_util import (assert_bf16_parity, assert_bytes_equal, dev_bf16, dev_f32, f32_bits, host,
                      require_gpu)
from helpers import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu

RSTD_ROUNDINGS = 32
EPS = 1e-6
FMTS = {"e4m3": ref.E4M3, "e5m2": ref.E5M2, "mx8": ref.MX8}


def draw(rng, rows, hidden, scale=1.0):
    x = rng.standard_normal((rows, hidden)).astype(np.float32)
    x *= np.exp(rng.standard_normal((rows, 1))).astype(np.float32) * np.float32(scale)
    return f32_to_bf16_bits(x)


def weight(rng, hidden, kind):
    w = (1 + 0.3 * rng.standard_normal(hidden)).astype(np.float32)
    return w if kind == "f32" else bf16_bits_to_f32(f32_to_bf16_bits(w))


def guarded(shape, dtype, dev):
    """An output with 64 sentinel bytes behind it, and the check of them."""
    n = int(np.prod(shape)) * dtype.itemsize
    raw = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device=dev)
    return raw[:n].view(dtype).view(shape), lambda: bool((raw[n:] == 0xA5).all())


def run(dev, fmt, xb, rb, w, kind, eps=EPS, want_y=True, in_place=False):
    """One norm into guarded outputs -> host arrays (q, scales, h, y, rstd)."""
    rows, hidden = xb.shape
    x = dev_bf16(xb, dev)
    res = None if rb is None else dev_bf16(rb, dev)
    wd = dev_f32(w, dev) if kind == "f32" else dev_bf16(f32_to_bf16_bits(w), dev)
    q, q_ok = guarded((rows, hidden), torch.uint8, dev)
    if fmt == ref.MX8:
        s, s_ok = guarded((rows, hidden // 32), torch.uint8, dev)
    else:
        s, s_ok = guarded((rows, -(-hidden // 128)), torch.float32, dev)
    rstd, r_ok = guarded((rows,), torch.float32, dev)
    y, y_ok = guarded((rows, hidden), torch.bfloat16, dev) if want_y else (None, lambda: True)
    h, h_ok = (None, lambda: True)
    if res is not None:
        h, h_ok = (res, lambda: True) if in_place else guarded((rows, hidden), torch.bfloat16, dev)
    kw = dict(residual=res, h_out=h, y_out=y, q_out=q, rstd_out=rstd)
    if fmt == ref.MX8:
        out = fq.mx8_rms_norm_quantize(x, wd, eps, e8m0_out=s, **kw)
    else:
        out = fq.fp8q_rms_norm_quantize(x, wd, eps, fmt=fmt, scales_out=s, **kw)
    torch.cuda.synchronize()
    assert out.q is q and out.scales is s and out.rstd is rstd
    assert q_ok() and s_ok() and r_ok() and y_ok() and h_ok(), "wrote past an output"
    return [None if t is None else host(t) for t in (q, s, h, y, rstd)]


def check(got, fmt, xb, rb, w, eps=EPS):
    q, s, h, y, rstd = got
    x = bf16_bits_to_f32(xb)
    r = None if rb is None else bf16_bits_to_f32(rb)
    _, rstd64, y64 = ref.rms_norm(x, r, w, eps)
    assert (np.abs(rstd - rstd64) <= RSTD_ROUNDINGS * ref.U32 * rstd64).all(), "rstd"
    h32, y32 = ref.norm_f32(x, r, w, rstd)
    codes, scales = ref.encode_rows(y32, fmt)
    assert_bytes_equal(q, codes, "codes")
    if fmt == ref.MX8:
        assert_bytes_equal(s, scales, "E8M0")
    else:
        assert_bytes_equal(f32_bits(s), f32_bits(scales), "scales")
    if h is not None:
        assert_bf16_parity(h, f32_to_bf16_bits(h32), "h")
    if y is not None:
        assert_bf16_parity(y, f32_to_bf16_bits(y32), "y")
    # and against 64 bits: y moves by rstd's error and two roundings more;
    # then half a step of the code, at most 2^-4 (e4m3) or 2^-3 (e5m2) of the
    # value, or half the smallest step; a code at the top may lose up to
    # 1 - 448/512 in MXFP8, whose scale is a power of two
    part = 32 if fmt == ref.MX8 else 128
    scale = ref.decode_rows(np.full_like(codes, 0x38 if fmt != ref.E5M2 else 0x3C), s, fmt)
    rel = {ref.E4M3: 2.0 ** -4, ref.E5M2: 2.0 ** -3, ref.MX8: 2.0 ** -3}[fmt]
    least = scale * {ref.E4M3: 2.0 ** -10, ref.E5M2: 2.0 ** -17, ref.MX8: 2.0 ** -10}[fmt]
    off = np.abs(ref.decode_rows(q, s, fmt) - y64)
    assert (off <= np.abs(y64) * (rel + (RSTD_ROUNDINGS + 8) * ref.U32) + least * 1.001).all(), part


HIDDEN = [1, 2, 7, 8, 9, 64, 127, 128, 129, 511, 512, 513, 768, 1000, 1411, 2048, 2049, 2888, 4096,
          4104, 6001, 8192, 8193, 16384, 20000, 32768]


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("hidden", HIDDEN)
def test_norm_blocks(hidden, fmt):
    dev = require_gpu()
    rng = np.random.default_rng(hidden)
    for rows, with_res, kind in [(1, True, "bf16"), (3, False, "f32"), (6, True, "f32"),
                                 (37 if hidden <= 4096 else 5, True, "bf16")]:
        xb = draw(rng, rows, hidden)
        rb = draw(rng, rows, hidden, 3.0) if with_res else None
        w = weight(rng, hidden, kind)
        check(run(dev, FMTS[fmt], xb, rb, w, kind, want_y=rows != 6), FMTS[fmt], xb, rb, w)


@pytest.mark.parametrize("hidden", [32, 64, 96, 160, 512, 544, 1024, 2048, 2080, 2912, 4096, 8192,
                                    16384, 32768])
def test_norm_mx8(hidden):
    dev = require_gpu()
    rng = np.random.default_rng(hidden)
    for rows, with_res, kind in [(1, True, "bf16"), (4, False, "f32"), (7, True, "f32")]:
        xb = draw(rng, rows, hidden)
        rb = draw(rng, rows, hidden, 3.0) if with_res else None
        w = weight(rng, hidden, kind)
        check(run(dev, ref.MX8, xb, rb, w, kind, want_y=rows != 4), ref.MX8, xb, rb, w)


@pytest.mark.parametrize("fmt", ["e4m3", "mx8"])
@pytest.mark.parametrize("rows,hidden", [(2050, 512), (4099, 1024), (1500, 2048), (700, 4096)])
def test_norm_many_rows(rows, hidden, fmt):
    dev = require_gpu()
    rng = np.random.default_rng(rows)
    xb, rb, w = draw(rng, rows, hidden), draw(rng, rows, hidden), weight(rng, hidden, "bf16")
    check(run(dev, FMTS[fmt], xb, rb, w, "bf16", in_place=True), FMTS[fmt], xb, rb, w)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2", "mx8"])
def test_norm_special_rows(fmt):
    """Zero rows, one element in a row, an inf, a NaN, values near the type's
    smallest and largest (whose squares leave fp32's range), tiny blocks in an
    ordinary row: the fp32 sequence decides, bit for bit."""
    dev = require_gpu()
    rng = np.random.default_rng(5)
    hidden = 640
    x = rng.standard_normal((12, hidden)).astype(np.float32)
    x[0] = 0
    x[1] = 0
    x[1, 333] = 3.0
    x[2, 7] = np.inf
    x[3, 500] = np.nan
    x[4, 0], x[4, 1] = np.inf, -np.inf
    x[5] = 1e-38
    x[6] *= np.float32(1e-40)
    x[7, 3] = 3e38
    x[8] *= np.float32(1e25)
    x[9, 128:256] *= np.float32(1e-30)
    x[10, 256:384] = -0.0
    x[11] = np.float32(2.0 ** -133)
    xb = f32_to_bf16_bits(x)
    w = weight(rng, hidden, "f32")
    w[600] = 0.0
    for eps in (EPS, 0.0):
        q, s, h, y, rstd = run(dev, FMTS[fmt], xb, None, w, "f32", eps=eps)
        xf = bf16_bits_to_f32(xb)
        with np.errstate(all="ignore"):
            _, rstd64, _ = ref.rms_norm(xf, None, w, eps)
        # rows whose sum of squares stays inside fp32's normal range (or is 0
        # with an eps above it)
        ss = (xf.astype(np.float64) ** 2).sum(1)
        plain = np.isfinite(ss) & (ss < 1e38) & ((ss > 1e-30) | (eps > 0))
        off = np.abs(rstd[plain] - rstd64[plain])
        assert (off <= RSTD_ROUNDINGS * ref.U32 * rstd64[plain]).all()
        assert np.isnan(rstd[3]) and rstd[2] == 0 and rstd[7] == 0 and rstd[8] == 0
        if eps == 0.0:
            assert np.isinf(rstd[0])
        h32, y32 = ref.norm_f32(xf, None, w, rstd)
        codes, scales = ref.encode_rows(y32, FMTS[fmt])
        assert_bytes_equal(q, codes, "codes")
        if fmt == "mx8":
            assert_bytes_equal(s, scales, "E8M0")
        else:
            assert np.array_equal(np.isnan(s), np.isnan(scales))
            assert_bytes_equal(f32_bits(s[~np.isnan(s)]), f32_bits(scales[~np.isnan(s)]), "scales")
        assert_bf16_parity(y, f32_to_bf16_bits(y32), "y")


@pytest.mark.parametrize("fmt", ["e4m3", "mx8"])
def test_norm_at_the_small_end_of_the_sum_of_squares(fmt):
    """Finite rows whose squares underflow in fp32: rstd inf, and no finite row
    out of it, with eps 0; an ordinary rstd with a small eps.  A row just above
    is normed as any other."""
    dev = require_gpu()
    hidden = 192
    x = np.zeros((4, hidden), np.float32)
    x[0] = 2.0 ** -76                          # squares of 2^-152 round to 0
    x[1, 7] = 2.0 ** -80
    x[2] = -(2.0 ** -100)
    x[3] = 2.0 ** -60                          # squares of 2^-120
    xb, w = f32_to_bf16_bits(x), np.ones(hidden, np.float32)
    q, s, _, y, rstd = run(dev, FMTS[fmt], xb, None, w, "f32", eps=0.0)
    assert np.isposinf(rstd[:3]).all() and abs(rstd[3] / 2.0 ** 60 - 1) <= RSTD_ROUNDINGS * ref.U32
    y = bf16_bits_to_f32(y)
    assert np.isposinf(y[0]).all() and np.isneginf(y[2]).all()
    assert np.isposinf(y[1, 7]) and np.isnan(np.delete(y[1], 7)).all()
    assert (q[:3] == 0x7F).all() and ((s[:3] == 255) if fmt == "mx8" else np.isnan(s[:3])).all()
    eps = 2.0 ** -100                          # about 8e-31
    got = run(dev, FMTS[fmt], xb, None, w, "f32", eps=eps)
    assert (np.abs(got[4][:3] / 2.0 ** 50 - 1) <= RSTD_ROUNDINGS * ref.U32).all()
    check(got, FMTS[fmt], xb, None, w, eps=eps)


def test_norm_reads_back_through_the_codec():
    """With hidden a multiple of 128 the rows are the codec's flat layout."""
    dev = require_gpu()
    rng = np.random.default_rng(9)
    xb = draw(rng, 10, 768)
    out = fq.fp8q_rms_norm_quantize(dev_bf16(xb, dev), torch.ones(768, device=dev))
    got = fq.fp8q_dequantize(out.q.reshape(-1), out.scales.reshape(-1), fq.E4M3)
    want = ref.decode_rows(host(out.q), host(out.scales), ref.E4M3)
    assert_bytes_equal(f32_bits(host(got)), f32_bits(want), "dequantize")
    mx = fq.mx8_rms_norm_quantize(dev_bf16(xb, dev), torch.ones(768, device=dev))
    got = fq.mx8_dequantize(mx.q, mx.scales)
    assert_bytes_equal(f32_bits(host(got)), f32_bits(ref.decode_rows(host(mx.q), host(mx.scales), ref.MX8)),
                       "mx8 dequantize")


def test_norm_of_nothing():
    dev = require_gpu()
    w = torch.ones(256, device=dev)
    out = fq.fp8q_rms_norm_quantize(torch.empty((0, 256), dtype=torch.bfloat16, device=dev), w)
    assert out.q.shape == (0, 256) and out.scales.shape == (0, 2)
    dx, dw = fq.fp8q_rms_norm_backward(torch.empty((0, 256), dtype=torch.bfloat16, device=dev),
                                       torch.empty((0, 256), dtype=torch.bfloat16, device=dev), w,
                                       torch.empty(0, device=dev))
    torch.cuda.synchronize()
    assert dx.shape == (0, 256) and (host(dw) == 0).all()


# --------------------------------------------------------------------------- #
# backward                                                                    #
# --------------------------------------------------------------------------- #

def grads(dev, dyb, hb, w, kind, rstd, dhb, in_place=None):
    rows, hidden = hb.shape
    dy, h = dev_bf16(dyb, dev), dev_bf16(hb, dev)
    dh = None if dhb is None else dev_bf16(dhb, dev)
    wd = dev_f32(w, dev) if kind == "f32" else dev_bf16(f32_to_bf16_bits(w), dev)
    dx, dx_ok = guarded((rows, hidden), torch.bfloat16, dev)
    if in_place is not None:
        dx, dx_ok = (dy if in_place == "dy" else dh), lambda: True
    dw, dw_ok = guarded((hidden,), torch.float32, dev)
    need = fq.fp8q_rms_norm_backward_workspace(rows, hidden)
    ws, ws_ok = guarded((need,), torch.uint8, dev)
    fq.fp8q_rms_norm_backward(dy, h, wd, dev_f32(rstd, dev), dh=dh, dx_out=dx, dweight_out=dw,
                              workspace=ws)
    torch.cuda.synchronize()
    assert dx_ok() and dw_ok() and ws_ok(), "wrote past an output"
    return bf16_bits_to_f32(host(dx)), host(dw)


def check_grads(got, dyb, hb, w, rstd, dhb):
    """dx: one rounding to bf16, and fp32 roundings of its three terms: the
    row's sum has at most 58 (as in the forward), its factors 6 more.  dw: a
    chain of at most `rows` additions and 4 roundings a term."""
    dx, dw = got
    dy, h = bf16_bits_to_f32(dyb).astype(np.float64), bf16_bits_to_f32(hb).astype(np.float64)
    dh = None if dhb is None else bf16_bits_to_f32(dhb)
    want_dx, want_dw = ref.rms_norm_grads(dy, h, w, rstd, dh)
    r = rstd.astype(np.float64)[:, None]
    g = np.abs(dy * w)
    c = r ** 3 * (g * np.abs(h)).sum(1, keepdims=True) / h.shape[1]
    mag = g * r + np.abs(h) * c + (0 if dh is None else np.abs(dh))
    assert (np.abs(dx - want_dx) <= ref.U16 * np.abs(want_dx) + 64 * ref.U32 * mag + ref.TINY16).all()
    mag = np.abs(dy * h * r).sum(0)
    assert (np.abs(dw - want_dw) <= (h.shape[0] + 4) * ref.U32 * mag).all()


@pytest.mark.parametrize("hidden", HIDDEN)
def test_norm_backward(hidden):
    dev = require_gpu()
    rng = np.random.default_rng(hidden)
    for rows, kind, with_dh in [(1, "f32", True), (2, "bf16", False), (35, "f32", True)]:
        hb, dyb = draw(rng, rows, hidden, 2.0), draw(rng, rows, hidden, 1e-2)
        dhb = draw(rng, rows, hidden, 1e-2) if with_dh else None
        w = weight(rng, hidden, kind)
        rstd = ref.rms_norm(bf16_bits_to_f32(hb), None, w, EPS)[1].astype(np.float32)
        check_grads(grads(dev, dyb, hb, w, kind, rstd, dhb), dyb, hb, w, rstd, dhb)


@pytest.mark.parametrize("rows,hidden", [(512, 72), (513, 72), (512, 1), (700, 1), (515, 7), (512, 9), (600, 9),
                                         (511, 513), (515, 513), (515, 1000), (512, 1411), (513, 1411),
                                         (509, 2888), (515, 2888), (515, 6001), (512, 8192), (515, 8192),
                                         (300, 16384), (515, 16384), (140, 32768), (515, 20000)])
def test_norm_backward_either_side_of_one_launch(rows, hidden):
    """Sizes around where one launch becomes two, at every way a row can end."""
    dev = require_gpu()
    rng = np.random.default_rng(rows + hidden)
    hb, dyb = draw(rng, rows, hidden, 2.0), draw(rng, rows, hidden, 1e-2)
    dhb = draw(rng, rows, hidden, 1e-2) if rows % 2 else None
    w = weight(rng, hidden, "f32" if rows % 3 else "bf16")
    kind = "f32" if rows % 3 else "bf16"
    rstd = ref.rms_norm(bf16_bits_to_f32(hb), None, w, EPS)[1].astype(np.float32)
    check_grads(grads(dev, dyb, hb, w, kind, rstd, dhb), dyb, hb, w, rstd, dhb)


@pytest.mark.parametrize("in_place", [None, "dy", "dh"])
@pytest.mark.parametrize("rows,hidden", [(1, 16392), (5, 32768), (700, 16385), (1300, 16392), (900, 20001)])
def test_norm_backward_wide_rows(rows, hidden, in_place):
    dev = require_gpu()
    rng = np.random.default_rng(7 * rows + hidden)
    hb, dyb, dhb = draw(rng, rows, hidden, 2.0), draw(rng, rows, hidden, 1e-2), draw(rng, rows, hidden, 1e-2)
    w = weight(rng, hidden, "f32")
    rstd = ref.rms_norm(bf16_bits_to_f32(hb), None, w, EPS)[1].astype(np.float32)
    check_grads(grads(dev, dyb, hb, w, "f32", rstd, dhb, in_place), dyb, hb, w, rstd, dhb)


@pytest.mark.parametrize("in_place", ["dy", "dh"])
@pytest.mark.parametrize("rows,hidden", [(1, 64), (3, 2048), (4, 9), (100, 513), (509, 2888), (512, 8192)])
def test_norm_backward_few_rows_in_place(rows, hidden, in_place):
    """dx over its own input: the weight's gradient still sees dy as it was."""
    dev = require_gpu()
    rng = np.random.default_rng(5 * rows + hidden)
    hb, dyb, dhb = draw(rng, rows, hidden, 2.0), draw(rng, rows, hidden, 1e-2), draw(rng, rows, hidden, 1e-2)
    w = weight(rng, hidden, "bf16")
    rstd = ref.rms_norm(bf16_bits_to_f32(hb), None, w, EPS)[1].astype(np.float32)
    got = grads(dev, dyb, hb, w, "bf16", rstd, dhb, in_place)
    check_grads(got, dyb, hb, w, rstd, dhb)
    again = grads(dev, dyb, hb, w, "bf16", rstd, dhb, in_place)
    assert all(np.array_equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("rows,hidden,in_place", [(1030, 512, "dh"), (2500, 1024, "dy"),
                                                  (1100, 2048, None), (1201, 4096, "dh"),
                                                  (5000, 72, None)])
def test_norm_backward_many_rows(rows, hidden, in_place):
    dev = require_gpu()
    rng = np.random.default_rng(rows)
    hb, dyb, dhb = (draw(rng, rows, hidden) for _ in range(3))
    w = weight(rng, hidden, "bf16")
    rstd = ref.rms_norm(bf16_bits_to_f32(hb), None, w, EPS)[1].astype(np.float32)
    first = grads(dev, dyb, hb, w, "bf16", rstd, dhb, in_place)
    check_grads(first, dyb, hb, w, rstd, dhb)
    again = grads(dev, dyb, hb, w, "bf16", rstd, dhb, in_place)
    assert all(np.array_equal(a, b) for a, b in zip(first, again)), "not the same bits twice"


@pytest.mark.parametrize("rows,hidden", [(1, 64), (3, 2048), (700, 2048), (600, 513), (3, 20000)])
@pytest.mark.parametrize("size,dy_size", [(1e-12, 1e-3), (1e-21, 1.0), (1e-25, 1e-3), (1e-33, 1e-2), (1e12, 1e-3),
                                          (1e17, 1.0)])
def test_norm_backward_of_rows_far_from_one(rows, hidden, size, dy_size):
    """Rows whose rstd^3 leaves fp32's range, with gradients whose products with
    them and whose dx are inside it."""
    dev = require_gpu()
    rng = np.random.default_rng(rows + hidden)
    hb, dyb = draw(rng, rows, hidden, size), draw(rng, rows, hidden, dy_size)
    w = weight(rng, hidden, "f32")
    rstd = ref.rms_norm(bf16_bits_to_f32(hb), None, w, 0.0)[1].astype(np.float32)
    assert np.isfinite(rstd).all() and (rstd > 0).all()
    check_grads(grads(dev, dyb, hb, w, "f32", rstd, None), dyb, hb, w, rstd, None)


def test_norm_backward_against_differences():
    """The device's gradients against central differences of the forward in
    64 bits, of loss = sum(dy * y) + sum(dh * h)."""
    dev = require_gpu()
    rng = np.random.default_rng(3)
    rows, hidden, eps = 3, 40, 1e-3
    hb, dyb, dhb = (draw(rng, rows, hidden) for _ in range(3))
    h, dy, dh = (bf16_bits_to_f32(b).astype(np.float64) for b in (hb, dyb, dhb))
    w = weight(rng, hidden, "f32")

    def loss(h_, w_):
        return (ref.rms_norm(h_, None, w_, eps)[2] * dy).sum() + (h_ * dh).sum()

    rstd = ref.rms_norm(h, None, w, eps)[1].astype(np.float32)
    dx, dw = grads(dev, dyb, hb, w, "f32", rstd, dhb)
    want_dx = ref.differences(lambda v: loss(v, w.astype(np.float64)), h, 1e-5)
    want_dw = ref.differences(lambda v: loss(h, v), w.astype(np.float64), 1e-5)
    # differences: about step^2 times a third derivative, 1e-8 here with room;
    # the device: a rounding to bf16 (dx), fp32 roundings of sums of order 10
    scale = np.abs(want_dx).max()
    assert np.abs(dx - want_dx).max() <= ref.U16 * scale + 1e-4
    assert np.abs(dw - want_dw).max() <= 1e-4
