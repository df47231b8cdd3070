"""Routing and its gradient on the GPU against 64 bits: the ids equal, weights
and gradients within the bounds that model_ref derives."""
import math

import numpy as np
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
import model_ref as ref
from gpu_util import host, require_gpu
from layer_ref import TINY16, U16

pytestmark = pytest.mark.gpu

# experts and topk on both sides of the kernels' shapes (lanes a token, logits a
# lane), tokens on both sides of a wave's and a workgroup's
SHAPES = [(1, 1, 1), (3, 5, 5), (1, 16, 8), (5, 17, 2), (17, 60, 6), (16, 64, 8), (1, 128, 8), (67, 128, 8),
          (33, 129, 4), (9, 128, 17), (9, 40, 33), (7, 256, 8), (5, 257, 8), (3, 512, 64), (3, 513, 8), (2, 1000, 7),
          (4, 1024, 64), (1025, 8, 2)]


def values(tokens, experts, dtype, seed, masked=0.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(tokens, experts, generator=g) * 3
    if masked:
        l[torch.rand(tokens, experts, generator=g) < masked] = -math.inf
    return l.to(dtype)


def close(got, want, bound, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what + ": NaN positions differ"
    ok = ~np.isnan(want)
    worst = (np.abs(got - want) - bound)[ok].max() if ok.any() else 0.0
    assert worst <= 0.0, "%s: %.3g past its bound" % (what, worst)


def forward(l, topk, normalize):
    dev = require_gpu()
    w, ids = fq.fp8q_moe_route(l.to(dev), topk, normalize=normalize)
    assert w.dtype == torch.float32 and ids.dtype == torch.int32 and w.shape == ids.shape == (l.shape[0], topk)
    return w, ids


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,topk", SHAPES)
def test_route_and_gradient(tokens, experts, topk, dtype, normalize):
    for masked in (0.0, 0.5):
        l = values(tokens, experts, dtype, 7 * tokens + experts + topk, masked)
        want, ids64, bound = ref.route(l.double().numpy(), topk, normalize)
        w, ids = forward(l, topk, normalize)
        assert np.array_equal(host(ids), ids64)
        close(host(w), want, bound, "weights")
        dw = torch.randn(tokens, topk, generator=torch.Generator().manual_seed(3))
        got = fq.fp8q_moe_route_backward(dw.to(w.device), l.to(w.device), w, ids, normalize=normalize)
        assert got.dtype == dtype and got.shape == l.shape
        d64, dbound = ref.route_grad(dw.numpy(), l.double().numpy(), host(w), host(ids), normalize)
        if dtype == torch.bfloat16:
            dbound = dbound + U16 * (np.abs(d64) + dbound) + TINY16
        close(got.double().cpu().numpy(), d64, dbound, "dlogits")


def test_ties_go_to_the_lowest_index():
    l = torch.zeros(6, 128)
    l[0] = 1.0
    l[1, ::2] = -0.0                    # equal to +0
    l[2] = torch.arange(128) // 4
    l[3, 100] = l[3, 7] = 5.0
    l[4] = -math.inf
    l[4, 90] = l[4, 60] = -3e38
    l[5] = 1e-45                        # subnormal, all equal
    w, ids = forward(l, 8, True)
    want, ids64, bound = ref.route(l.numpy(), 8, True)
    assert host(ids)[0].tolist() == list(range(8)) and host(ids)[1].tolist() == list(range(8))
    assert host(ids)[4].tolist() == [60, 90] + [-1] * 6
    assert np.array_equal(host(ids), ids64)
    close(host(w), want, bound, "weights")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [True, False])
def test_rows_without_experts_and_special_values(normalize, dtype):
    l = values(9, 60, dtype, 5)
    l[0] = -math.inf                    # nothing to choose
    l[1, 1:] = -math.inf                # one expert, for four choices
    l[2, 17] = math.inf
    l[3, 40] = math.nan
    l[3, 20] = math.inf
    l[4, 30] = l[4, 12] = math.nan
    l[5, :] = torch.finfo(dtype).min    # the type's lowest value is a logit as any
    l[6, :] = torch.finfo(dtype).min
    l[6, 33] = torch.finfo(dtype).max
    w, ids = forward(l, 4, normalize)
    want, ids64, bound = ref.route(l.double().numpy(), 4, normalize)
    assert np.array_equal(host(ids), ids64)
    assert host(ids)[0].tolist() == [-1] * 4 and not host(w)[0].any()
    assert host(ids)[1].tolist() == [0, -1, -1, -1] and host(w)[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert host(ids)[3].tolist()[:2] == [40, 20] and host(ids)[4].tolist()[:2] == [12, 30]
    assert np.isnan(host(w)[2:5]).all()
    close(host(w)[[0, 1, 5, 6, 7, 8]], want[[0, 1, 5, 6, 7, 8]], bound[[0, 1, 5, 6, 7, 8]], "weights")
    dw = torch.full((9, 4), 0.5)
    dw[0] = math.nan                    # of choices that are none: not used
    dw[1, 1:] = math.nan
    d = fq.fp8q_moe_route_backward(dw.to(w.device), l.to(w.device), w, ids, normalize=normalize)
    d64, dbound = ref.route_grad(np.nan_to_num(dw.numpy()), l.double().numpy(), host(w), host(ids), normalize)
    got = d.double().cpu().numpy()
    assert not got[0].any()
    for t in (0, 1, 5, 6, 7, 8):
        close(got[t], d64[t], dbound[t] + (U16 * (np.abs(d64[t]) + dbound[t]) + TINY16 if dtype == torch.bfloat16 else 0),
              "dlogits %d" % t)


def test_gradient_of_foreign_and_repeated_ids():
    """Ids that did not come from the routing: outside the experts, and one
    expert twice (its gradients add up)."""
    dev = require_gpu()
    l = values(3, 32, torch.float32, 2)
    ids = torch.tensor([[3, 3, 40, -7], [31, 0, 31, 31], [2 ** 31 - 1, -2 ** 31, 5, 5]], dtype=torch.int32)
    w = torch.rand(3, 4, generator=torch.Generator().manual_seed(1))
    dw = torch.randn(3, 4, generator=torch.Generator().manual_seed(2))
    for normalize in (True, False):
        d = fq.fp8q_moe_route_backward(dw.to(dev), l.to(dev), w.to(dev), ids.to(dev), normalize=normalize)
        d64, bound = ref.route_grad(dw.numpy(), l.numpy(), w.numpy(), ids.numpy(), normalize)
        close(host(d), d64, bound, "dlogits")


@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(normalize):
    """The 64-bit gradient that the kernel is held to is the derivative of the
    64-bit routing (the choice fixed)."""
    from layer_ref import differences
    l = values(2, 12, torch.float32, 4).double().numpy()
    w, ids, _ = ref.route(l, 3, normalize)
    dw = np.random.default_rng(0).normal(size=(2, 3))

    def loss(x):
        e = np.exp(x - x.max(1, keepdims=True))
        part = np.take_along_axis(e, ids, 1)
        return float((part / (part if normalize else e).sum(1, keepdims=True) * dw).sum())
    d64, _ = ref.route_grad(dw, l, w, ids, normalize)
    assert np.abs(differences(loss, l, 1e-6) - d64).max() < 1e-8


def test_in_place_repeats_and_given_outputs():
    dev = require_gpu()
    l = values(100, 96, torch.float32, 9).to(dev)
    w, ids = fq.fp8q_moe_route(l, 5)
    w2 = torch.full((101, 5), 7.0, device=dev)
    i2 = torch.full((101, 5), 7, dtype=torch.int32, device=dev)
    got = fq.fp8q_moe_route(l, 5, weights_out=w2[:100], ids_out=i2[:100])
    assert got[0].data_ptr() == w2.data_ptr() and torch.equal(w2[:100], w) and torch.equal(i2[:100], ids)
    assert (w2[100] == 7).all() and (i2[100] == 7).all()
    dw = torch.randn(100, 5, device=dev)
    for normalize in (True, False):
        want = fq.fp8q_moe_route_backward(dw, l, w, ids, normalize=normalize)
        buf = torch.cat([l, torch.full((1, 96), 3.0, device=dev)])
        got = fq.fp8q_moe_route_backward(dw, buf[:100], w, ids, normalize=normalize, dlogits_out=buf[:100])
        assert got.data_ptr() == buf.data_ptr() and torch.equal(buf[:100], want) and (buf[100] == 3).all()
    e = torch.zeros(0, 96, device=dev)
    w0, i0 = fq.fp8q_moe_route(e, 5)
    assert w0.shape == (0, 5) and fq.fp8q_moe_route_backward(w0, e, w0, i0).shape == (0, 96)


def test_the_sort_takes_a_routing_with_padding():
    l = values(40, 16, torch.float32, 11, 0.8).to(require_gpu())
    w, ids = fq.fp8q_moe_route(l, 4)
    slots, pairs, offsets = fq.fp8q_moe_sort(ids, 16)
    assert torch.equal(slots >= 0, ids >= 0) and int(offsets[-1]) == int((ids >= 0).sum())
    assert not w[ids < 0].any()


def test_refusals():
    dev = require_gpu()
    l = torch.zeros(4, 8, device=dev)
    w, ids = torch.zeros(4, 2, device=dev), torch.zeros(4, 2, dtype=torch.int32, device=dev)
    for bad in (lambda: fq.fp8q_moe_route(l, 0), lambda: fq.fp8q_moe_route(l, 9), lambda: fq.fp8q_moe_route(l[0], 2),
                lambda: fq.fp8q_moe_route(torch.zeros(4, 1025, device=dev), 2),
                lambda: fq.fp8q_moe_route(l.T, 2), lambda: fq.fp8q_moe_route(l, 2, weights_out=w[:3]),
                lambda: fq.fp8q_moe_route_backward(w, l[:3], w, ids),
                lambda: fq.fp8q_moe_route_backward(w, l, w[:3], ids),
                lambda: fq.fp8q_moe_route_backward(w, l, w, ids[:, :1]),
                lambda: fq.fp8q_moe_route_backward(w, l, w, ids, dlogits_out=l[:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fq.fp8q_moe_route(l.double(), 2), lambda: fq.fp8q_moe_route(l, 2.5),
                lambda: fq.fp8q_moe_route(l, 2, ids_out=ids.long()),
                lambda: fq.fp8q_moe_route(l, 2, normalize=torch.ones(2)),
                lambda: fq.fp8q_moe_route_backward(w, l, w, ids.long()),
                lambda: fq.fp8q_moe_route_backward(w, l, w, ids, dlogits_out=l.bfloat16())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_moe_route(l, 2, weights_out=l.view(-1)[:8].view(4, 2))


@pytest.mark.parametrize("normalize", [True, False])
def test_gradients_in_the_logits_place_are_a_change_to_autograd(normalize):
    dev = require_gpu()
    x = torch.randn(6, 8, device=dev, requires_grad=True)
    logits = x * 2.0
    loss = (logits * logits).sum()          # saves the logits
    weights, ids = fq.fp8q_moe_route(logits.detach(), 2, normalize=normalize)
    want = fq.fp8q_moe_route_backward(torch.ones_like(weights), logits.detach(), weights, ids, normalize=normalize)
    version = logits._version
    got = fq.fp8q_moe_route_backward(torch.ones_like(weights), logits.detach(), weights, ids, normalize=normalize,
                                     dlogits_out=logits.detach())
    assert torch.equal(got, want) and logits._version == version + 1
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
