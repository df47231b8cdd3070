"""The sort, permute, combine and its gradient against the plain forms of
layer_ref: integers and copied bytes equal, sums within derived bounds of 64
bits.  Outputs have sentinels behind them."""
import numpy as np
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
import layer_ref as ref
from gpu_util import dev_bf16, dev_f32, dev_u8, host, require_gpu
from helpers import bf16_bits_to_f32, f32_to_bf16_bits
from test_gpu_rms_norm import guarded

pytestmark = pytest.mark.gpu


def dev_ids(ids, dev, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(ids)).to(dev).to(dtype)


def choose(rng, tokens, topk, experts, dropped=0.0):
    """Distinct experts a token (where there are enough), some dropped."""
    score = rng.random((tokens, experts)) * (0.2 + rng.random(experts))
    ids = np.argsort(-score, axis=1)[:, :topk].astype(np.int32)
    if topk > experts:
        ids = rng.integers(0, experts, (tokens, topk)).astype(np.int32)
    if dropped:
        ids[rng.random(ids.shape) < dropped] = -1
        ids[rng.random(tokens) < dropped] = experts + 5
    return ids


def sort_on(dev, ids, experts, dtype=torch.int32):
    tokens, topk = ids.shape
    slots, a = guarded((tokens, topk), torch.int32, dev)
    pairs, b = guarded((tokens * topk,), torch.int32, dev)
    offsets, c = guarded((experts + 1,), torch.int32, dev)
    need = fq.fp8q_moe_sort_workspace(tokens, topk, experts)
    ws, d = guarded((need,), torch.uint8, dev)
    fq.fp8q_moe_sort(dev_ids(ids, dev, dtype), experts, slots_out=slots, pairs_out=pairs,
                     offsets_out=offsets, workspace=ws)
    torch.cuda.synchronize()
    assert a() and b() and c() and d(), "wrote past an output"
    return host(slots), host(pairs), host(offsets)


def check_sort(dev, ids, experts, dtype=torch.int32):
    for got, want, what in zip(sort_on(dev, ids, experts, dtype), ref.moe_sort(ids, experts),
                               ("slots", "pairs", "offsets")):
        assert np.array_equal(got, want), what


@pytest.mark.parametrize("experts", [1, 2, 60, 64, 128, 257, 1024])
@pytest.mark.parametrize("tokens,topk", [(1, 1), (1, 8), (3, 5), (64, 1), (65, 2), (129, 8),
                                         (1000, 6), (2049, 8), (5000, 4)])
def test_sort(tokens, topk, experts):
    dev = require_gpu()
    rng = np.random.default_rng(tokens + experts)
    check_sort(dev, choose(rng, tokens, topk, experts), experts)
    check_sort(dev, choose(rng, tokens, topk, experts, 0.3), experts, torch.int64)


@pytest.mark.parametrize("tokens,topk,experts", [(16383, 8, 128), (200000, 2, 60), (70001, 16, 1024),
                                                 (1 << 20, 1, 7), (2048, 64, 256), (300001, 8, 128)])
def test_sort_many_pairs(tokens, topk, experts):
    dev = require_gpu()
    rng = np.random.default_rng(tokens)
    ids = rng.integers(-1, experts + 1, (tokens, topk)).astype(np.int32)
    check_sort(dev, ids, experts)


@pytest.mark.parametrize("tokens", [40, 4000, 40000])
def test_sort_one_expert_for_all_and_none(tokens):
    dev = require_gpu()
    check_sort(dev, np.full((tokens, 4), 17, np.int32), 32)
    check_sort(dev, np.full((tokens, 4), -1, np.int32), 32)
    check_sort(dev, np.full((tokens, 4), 32, np.int32), 32)
    wild = np.array([2 ** 31 - 1, -2 ** 31, 0, 31], np.int32)
    check_sort(dev, np.tile(wild, (tokens, 1)), 32)
    far = np.array([2 ** 32, 2 ** 32 + 3, -2 ** 63, 5], np.int64)
    check_sort(dev, np.tile(far, (tokens, 1)), 32, torch.int64)


def test_sort_of_nothing():
    dev = require_gpu()
    offsets = torch.full((9,), 7, dtype=torch.int32, device=dev)
    slots, pairs, _ = fq.fp8q_moe_sort(torch.empty((0, 4), dtype=torch.int32, device=dev), 8,
                                       offsets_out=offsets)
    torch.cuda.synchronize()
    assert slots.shape == (0, 4) and pairs.shape == (0,) and (host(offsets) == 0).all()


# --------------------------------------------------------------------------- #

def slot_table(rng, tokens, topk, rows, dropped):
    """Distinct slots of a buffer of `rows` rows, in no order, some -1."""
    n = tokens * topk
    slots = rng.permutation(max(rows, n))[:n].astype(np.int32)
    slots[slots >= rows] = -1
    slots[rng.random(n) < dropped] = -1
    return slots.reshape(tokens, topk)


@pytest.mark.parametrize("row_bytes", [1, 2, 15, 16, 17, 64, 127, 1000, 1024, 1025, 2048, 2822, 4096,
                                       16384, 33000])
def test_permute_bytes(row_bytes):
    dev = require_gpu()
    rng = np.random.default_rng(row_bytes)
    for tokens, topk, dropped, scale_bytes in [(1, 8, 0.0, 64), (5, 1, 0.0, 1), (33, 6, 0.3, 7),
                                               (70, 3, 0.5, 2300), (9, 64, 0.2, 0)]:
        rows = tokens * topk
        slots = slot_table(rng, tokens, topk, rows, dropped)
        x = rng.integers(0, 256, (tokens, row_bytes), dtype=np.uint8)
        s = rng.integers(0, 256, (tokens, scale_bytes), dtype=np.uint8) if scale_bytes else None
        out, ok = guarded((rows, row_bytes), torch.uint8, dev)
        sout, sok = guarded((rows, scale_bytes), torch.uint8, dev) if scale_bytes else (None, lambda: True)
        fq.fp8q_moe_permute(dev_u8(x, dev), torch.from_numpy(slots).to(dev),
                            scales=None if s is None else dev_u8(s, dev), out=out, scales_out=sout)
        torch.cuda.synchronize()
        assert ok() and sok(), "wrote past an output"
        want = np.full((rows, row_bytes), 0xA5, np.uint8)      # rows no slot names stay
        held = slots >= 0
        token = np.broadcast_to(np.arange(tokens)[:, None], slots.shape)
        want[slots[held]] = x[token[held]]
        assert np.array_equal(host(out), want)
        if s is not None:
            want = np.full((rows, scale_bytes), 0xA5, np.uint8)
            want[slots[held]] = s[token[held]]
            assert np.array_equal(host(sout), want)


def test_permute_skips_slots_outside_the_buffer():
    dev = require_gpu()
    x = torch.arange(6, dtype=torch.float32, device=dev).reshape(3, 2).to(torch.bfloat16)
    slots = torch.tensor([[0, 4], [2 ** 31 - 1, 1], [-2 ** 31, 3]], dtype=torch.int32, device=dev)
    out = torch.full((4, 2), 9.0, dtype=torch.bfloat16, device=dev)
    fq.fp8q_moe_permute(x, slots, out=out)
    torch.cuda.synchronize()
    assert out.float().cpu().tolist() == [[0, 1], [2, 3], [9, 9], [4, 5]]


def rows_of(rng, n, hidden, fmt, dev):
    """Expert rows of a format: device tensors (rows, scales) and fp32 values."""
    if fmt == "bf16":
        b = f32_to_bf16_bits(rng.standard_normal((n, hidden)).astype(np.float32))
        return dev_bf16(b, dev), None, bf16_bits_to_f32(b)
    code = {"e4m3": ref.E4M3, "e5m2": ref.E5M2, "mx8": ref.MX8}[fmt]
    q, s = ref.encode_rows(rng.standard_normal((n, hidden)).astype(np.float32)
                           * np.exp(rng.standard_normal((n, 1))).astype(np.float32), code)
    return (dev_u8(q, dev), dev_u8(s, dev) if fmt == "mx8" else dev_f32(s, dev),
            ref.decode_rows(q, s, code))


def combine_on(dev, rows, scales, slots, weights, fmt, out_dtype):
    tokens, hidden = slots.shape[0], rows.shape[1]
    out, ok = guarded((tokens, hidden), out_dtype, dev)
    fq.fp8q_moe_combine(rows, torch.from_numpy(slots).to(dev),
                        None if weights is None else dev_f32(weights, dev), scales=scales,
                        fmt=fq.E5M2 if fmt == "e5m2" else fq.E4M3, out_dtype=out_dtype, out=out)
    torch.cuda.synchronize()
    assert ok(), "wrote past the output"
    return host(out) if out_dtype == torch.float32 else bf16_bits_to_f32(host(out))


def check_combine(got, values, slots, weights, out_dtype):
    """topk fused multiply-adds: at most topk roundings of a partial sum no
    larger than the sum of magnitudes; then one to bf16."""
    want, mag = ref.combine(values, slots, weights)
    lim = slots.shape[1] * ref.U32 * mag * 1.01
    if out_dtype == torch.bfloat16:
        lim = lim + ref.U16 * np.abs(want) + ref.TINY16
    assert (np.abs(got - want) <= lim).all()
    assert (got[(slots < 0).all(1)] == 0).all()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "e5m2", "mx8"])
@pytest.mark.parametrize("hidden", [1, 8, 32, 72, 128, 331, 512, 768, 1000, 2048, 2049, 4096, 9000])
def test_combine(hidden, fmt):
    if fmt == "mx8":
        hidden = max(32, hidden // 32 * 32)
    dev = require_gpu()
    rng = np.random.default_rng(hidden)
    for tokens, topk, dropped, weighted, out_dtype in [
            (1, 8, 0.0, True, torch.bfloat16), (7, 1, 0.0, False, torch.float32),
            (21, 6, 0.4, True, torch.float32), (40, 4, 0.2, False, torch.bfloat16),
            (3, 64, 0.1, True, torch.float32), (11, 9, 0.0, True, torch.bfloat16)]:
        n = tokens * topk
        rows, scales, values = rows_of(rng, n, hidden, fmt, dev)
        slots = slot_table(rng, tokens, topk, n, dropped)
        slots[-1] = -1 if dropped else slots[-1]
        weights = rng.random((tokens, topk)).astype(np.float32) if weighted else None
        got = combine_on(dev, rows, scales, slots, weights, fmt, out_dtype)
        check_combine(got, values, slots, weights, out_dtype)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "mx8"])
def test_combine_does_not_read_what_no_slot_names(fmt):
    """NaN and inf in rows without a slot, and in the weights of pairs without
    one, stay out of every sum; one in a named row reaches its token alone."""
    dev = require_gpu()
    rng = np.random.default_rng(4)
    rows, scales, values = rows_of(rng, 12, 256, fmt, dev)
    slots = np.array([[0, 3], [-1, 5], [-1, -1], [7, 12], [2 ** 30, 8]], np.int32)
    weights = rng.random((5, 2)).astype(np.float32)
    weights[1, 0], weights[2] = np.nan, np.inf
    bad = [1, 2, 4, 6, 9, 10, 11]
    if fmt == "bf16":
        rows[bad] = float("nan")
        rows[8, 17] = float("inf")
    else:
        rows[bad] = 0x7F
        scales[bad] = 255 if fmt == "mx8" else float("inf")
        rows[8, 17] = 0x7F
    got = combine_on(dev, rows, scales, slots, weights, fmt, torch.float32)
    assert np.isfinite(got[:4]).all() and (got[2] == 0).all()
    assert not np.isfinite(got[4, 17]) and np.isfinite(np.delete(got[4], 17)).all()
    check_combine(got[:4], values, slots[:4], weights[:4], torch.float32)


def test_combine_of_nothing():
    dev = require_gpu()
    empty = torch.empty((0, 64), dtype=torch.bfloat16, device=dev)
    out = fq.fp8q_moe_combine(empty, torch.full((3, 2), -1, dtype=torch.int32, device=dev))
    torch.cuda.synchronize()
    assert out.shape == (3, 64) and (out == 0).all()
    out = fq.fp8q_moe_combine(torch.ones((4, 64), dtype=torch.bfloat16, device=dev),
                              torch.empty((0, 2), dtype=torch.int32, device=dev))
    assert out.shape == (0, 64)


def grads_on(dev, dyb, rb, slots, weights):
    drows, a = guarded(rb.shape, torch.bfloat16, dev)
    dw, b = guarded(slots.shape, torch.float32, dev)
    fq.fp8q_moe_combine_backward(dev_bf16(dyb, dev), dev_bf16(rb, dev), torch.from_numpy(slots).to(dev),
                                 dev_f32(weights, dev), drows_out=drows, dweights_out=dw)
    torch.cuda.synchronize()
    assert a() and b(), "wrote past an output"
    return host(drows), host(dw)


@pytest.mark.parametrize("hidden", [1, 7, 8, 72, 128, 512, 513, 1411, 2048, 4096, 9000])
def test_combine_backward(hidden):
    """drows: one product rounded to fp32 and once to bf16.  dweights: a chain
    of at most hidden fused multiply-adds and the wave's 6 (the bound holds
    for every order of the sum)."""
    dev = require_gpu()
    rng = np.random.default_rng(hidden)
    for tokens, topk, dropped in [(1, 8, 0.0), (13, 6, 0.4), (5, 1, 0.0), (3, 64, 0.1), (6, 11, 0.2)]:
        n = tokens * topk
        rb = f32_to_bf16_bits(rng.standard_normal((n, hidden)).astype(np.float32))
        dyb = f32_to_bf16_bits(rng.standard_normal((tokens, hidden)).astype(np.float32))
        slots = slot_table(rng, tokens, topk, n, dropped)
        weights = rng.random((tokens, topk)).astype(np.float32)
        drows, dw = grads_on(dev, dyb, rb, slots, weights)
        want, want_dw, mag = ref.combine_grads(bf16_bits_to_f32(dyb), bf16_bits_to_f32(rb), slots, weights)
        named = ~np.isnan(want).any(1)
        got = bf16_bits_to_f32(drows)
        lim = (ref.U16 + 2 * ref.U32) * np.abs(want[named]) + ref.TINY16
        assert (np.abs(got[named] - want[named]) <= lim).all()
        assert (drows[~named] == 0xA5A5).all(), "a row that no slot names was written"
        assert (np.abs(dw - want_dw) <= (hidden + 6) * ref.U32 * mag).all()
        assert (dw[slots < 0] == 0).all()


@pytest.mark.parametrize("tokens,topk,hidden", [(1100, 8, 2048), (5000, 4, 72), (1301, 2, 1000), (2300, 1, 331)])
def test_combine_and_its_gradient_in_large_grids(tokens, topk, hidden):
    """More than 512 workgroups, and no multiple of that: from there on they take
    tokens in runs an XCD, and the rest in their own order."""
    dev = require_gpu()
    rng = np.random.default_rng(tokens)
    n = tokens * topk
    slots = slot_table(rng, tokens, topk, n, 0.1)
    weights = rng.random((tokens, topk)).astype(np.float32)
    for fmt in ("bf16", "e4m3"):
        rows, scales, values = rows_of(rng, n, hidden, fmt, dev)
        check_combine(combine_on(dev, rows, scales, slots, weights, fmt, torch.float32), values, slots, weights,
                      torch.float32)
    rb = f32_to_bf16_bits(rng.standard_normal((n, hidden)).astype(np.float32))
    dyb = f32_to_bf16_bits(rng.standard_normal((tokens, hidden)).astype(np.float32))
    drows, dw = grads_on(dev, dyb, rb, slots, weights)
    want, want_dw, mag = ref.combine_grads(bf16_bits_to_f32(dyb), bf16_bits_to_f32(rb), slots, weights)
    named = ~np.isnan(want).any(1)
    off = np.abs(bf16_bits_to_f32(drows)[named] - want[named])
    assert (off <= (ref.U16 + 2 * ref.U32) * np.abs(want[named]) + ref.TINY16).all()
    assert (drows[~named] == 0xA5A5).all(), "a row that no slot names was written"
    assert (np.abs(dw - want_dw) <= (hidden + 6) * ref.U32 * mag).all()


def test_combine_backward_against_differences():
    dev = require_gpu()
    rng = np.random.default_rng(8)
    tokens, topk, hidden = 4, 3, 24
    rb = f32_to_bf16_bits(rng.standard_normal((12, hidden)).astype(np.float32))
    dyb = f32_to_bf16_bits(rng.standard_normal((tokens, hidden)).astype(np.float32))
    slots = slot_table(rng, tokens, topk, 12, 0.2)
    weights = rng.random((tokens, topk)).astype(np.float32)
    dy = bf16_bits_to_f32(dyb).astype(np.float64)
    drows, dw = grads_on(dev, dyb, rb, slots, weights)
    r64, w64 = bf16_bits_to_f32(rb).astype(np.float64), weights.astype(np.float64)

    def loss(r_, w_):
        out = np.zeros((tokens, hidden))
        for t in range(tokens):
            for j in range(topk):
                if slots[t, j] >= 0:
                    out[t] += w_[t, j] * r_[slots[t, j]]
        return (out * dy).sum()

    want = ref.differences(lambda v: loss(v, w64), r64, 1e-4)
    named = np.isin(np.arange(12), slots)
    # the loss is linear in each argument: differences are exact to 64-bit
    # cancellation, about 1e-11 here
    assert np.abs(bf16_bits_to_f32(drows)[named] - want[named]).max() <= ref.U16 * np.abs(want).max() + 1e-6
    want = ref.differences(lambda v: loss(r64, v), w64, 1e-4)
    assert np.abs(dw - want).max() <= 1e-4


def test_permutes_gradient_is_combine_with_ones():
    """sum(permute(x) * d) differentiated by x: each token's d rows, summed."""
    dev = require_gpu()
    rng = np.random.default_rng(11)
    ids = choose(rng, 50, 4, 16, 0.2)
    slots, pairs, offsets = fq.fp8q_moe_sort(dev_ids(ids, dev), 16)
    d = f32_to_bf16_bits(rng.standard_normal((200, 136)).astype(np.float32))
    got = host(fq.fp8q_moe_combine(dev_bf16(d, dev), slots, out_dtype=torch.float32))
    want, mag = ref.combine(bf16_bits_to_f32(d), ref.moe_sort(ids, 16)[0], None)
    assert (np.abs(got - want) <= 4 * ref.U32 * mag * 1.01).all()
