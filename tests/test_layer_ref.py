"""The plain forms that the layer operators are tested against: their
gradients against central differences of their own forward in 64 bits, their
encode against the oracle's quantize where both take bf16 values."""
import numpy as np
import pytest

import layer_ref as ref
import oracle
from helpers import bf16_bits_to_f32, f32_to_bf16_bits


def test_norm_gradients_against_differences():
    rng = np.random.default_rng(0)
    x, dy, dh = (rng.standard_normal((3, 11)) for _ in range(3))
    w = 1 + 0.2 * rng.standard_normal(11)
    eps = 1e-3

    def loss(x_, w_):
        h, _, y = ref.rms_norm(x_, None, w_, eps)
        return (y * dy).sum() + (h * dh).sum()

    h, rstd, _ = ref.rms_norm(x, None, w, eps)
    dx, dw = ref.rms_norm_grads(dy, h, w, rstd, dh)
    # central differences: error of the order step^2 = 1e-10 against values of order 1
    assert np.abs(dx - ref.differences(lambda v: loss(v, w), x, 1e-5)).max() < 1e-8
    assert np.abs(dw - ref.differences(lambda v: loss(x, v), w, 1e-5)).max() < 1e-8


def test_combine_gradients_against_differences():
    rng = np.random.default_rng(1)
    slots = np.array([[2, 0], [-1, 4], [1, -1], [-1, -1]])
    rows, w, dy = rng.standard_normal((5, 7)), rng.random((4, 2)), rng.standard_normal((4, 7))

    def loss(r_, w_):
        out = np.zeros((4, 7))
        for t in range(4):
            for j in range(2):
                if slots[t, j] >= 0:
                    out[t] += w_[t, j] * r_[slots[t, j]]
        return (out * dy).sum()

    drows, dw, _ = ref.combine_grads(dy, rows, slots, w)
    want = ref.differences(lambda v: loss(v, w), rows, 1e-4)
    named = [0, 1, 2, 4]
    assert np.abs(drows[named] - want[named]).max() < 1e-10 and np.isnan(drows[3]).all()
    assert np.abs(dw - ref.differences(lambda v: loss(rows, v), w, 1e-4)).max() < 1e-10


@pytest.mark.parametrize("fmt", [ref.E4M3, ref.E5M2, ref.MX8])
def test_encode_equals_the_oracles_quantize_on_bf16_values(fmt):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((6, 256)).astype(np.float32) * np.exp(rng.standard_normal((6, 1)) * 20).astype(np.float32)
    x[1] = 0
    x[2, 5], x[3, 130] = np.inf, np.nan
    x[4] *= np.float32(2.0 ** -100)
    bits = f32_to_bf16_bits(x)
    codes, scales = ref.encode_rows(bf16_bits_to_f32(bits), fmt)
    if fmt == ref.MX8:
        q, s = oracle.mx8_quantize(bits)
        assert np.array_equal(scales, s)
    else:
        q, s = oracle.quantize(bits, fmt)
        s = s.reshape(6, 2)
        assert np.array_equal(np.isnan(scales), np.isnan(s))
        assert np.array_equal(scales[~np.isnan(s)], s[~np.isnan(s)])
    assert np.array_equal(codes, q.reshape(6, 256))


def test_sort_of_a_small_table():
    ids = np.array([[2, 0], [0, 5], [-1, 2]])
    slots, pairs, offsets = ref.moe_sort(ids, 4)
    assert slots.tolist() == [[2, 0], [1, -1], [-1, 3]]
    assert pairs.tolist() == [1, 2, 0, 5, -1, -1]
    assert offsets.tolist() == [0, 2, 2, 4, 4]
