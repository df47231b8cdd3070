"""The model's operators as a program uses them: together along the wire,
captured in HIP graphs, on named streams, from several threads, and in grids
that have to be split."""
import ctypes
import math
import os
import threading

import pytest
import torch

import dequantize_reduce_transfer_amd as fq
import model_ref as ref
from dequantize_reduce_transfer_amd import model
from gpu_util import require_gpu
from stream_fakes import FakeStreams, logged, recorded

HERE = os.path.dirname(os.path.abspath(__file__))
E, I, H, K = 16, 192, 288, 4


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def inputs(dev, tokens, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    d = dict(x=rand(tokens, H).bfloat16(), logits=rand(tokens, E) * 2, dweights=rand(tokens, K),
             grads=[rand(n) for n in (3, 7001, 1 << 17)] + [rand(5001).bfloat16()])
    for k, (r, c) in dict(gate=(I, H), up=(I, H), down=(H, I)).items():
        d[k], d[k + "_scales"] = fq.mx8_quantize((rand(E, r, c) * c ** -0.5).bfloat16())
    return d


def chain(d, stream=None):
    """Every entry point once; the gradients' copies are clipped."""
    kw = dict(stream=stream)
    weights, ids = fq.fp8q_moe_route(d["logits"], K, **kw)
    dlogits = fq.fp8q_moe_route_backward(d["dweights"], d["logits"], weights, ids, **kw)
    plain, pids = fq.fp8q_moe_route(d["logits"], K, normalize=False, **kw)
    dplain = fq.fp8q_moe_route_backward(d["dweights"], d["logits"], plain, pids, normalize=False, **kw)
    m = [d[k] for k in ("gate", "up", "down")]
    s = {k + "_scales": d[k + "_scales"] for k in ("gate", "up", "down")}
    y = fq.fp8q_moe_experts(d["x"], ids, weights, *m, **s, **kw)
    y32 = fq.fp8q_moe_experts(d["x"], ids, weights, *m, **s, out_dtype=torch.float32, **kw)
    sumsq = fq.fp8q_grad_sumsq(d["grads"], **kw)
    small = fq.fp8q_grad_sumsq(d["grads"][:2], **kw)
    return [weights, ids, dlogits, plain, pids, dplain, y, y32, sumsq, small]


@pytest.mark.gpu
@pytest.mark.parametrize("tokens", [1, 5, 40, 200])
def test_graph_replays_equal_eager(tokens):
    """One token, a few, and numbers on both sides of the few-pair kernels;
    replays between other work, on new inputs in the captured buffers."""
    dev = require_gpu()
    d = inputs(dev, tokens)
    chain(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain(d)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(d)
    for seed in range(4):
        new = inputs(dev, tokens, seed)
        for k, v in d.items():
            for a, b in zip(v, new[k]) if isinstance(v, list) else [(v, new[k])]:
                a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = chain(new)
        assert all(same(a, b) for a, b in zip(got, want))
        graph.replay()
        assert all(same(a, b) for a, b in zip(out, want))


@pytest.mark.gpu
def test_clipping_in_a_graph():
    """The norm and the clipping captured together: each replay clips what is in
    the buffers then."""
    dev = require_gpu()
    g = [torch.zeros(n, device=dev) for n in (100, 70001)]

    def step():
        s = fq.fp8q_grad_sumsq(g)
        return fq.fp8q_grad_clip(g, s, 1.0, eps=0.0)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    for scale in (0.5, 0.0001, 3.0):
        for t in g:
            t.fill_(scale)
        graph.replay()
        torch.cuda.synchronize()
        want = scale * math.sqrt(70101)
        assert abs(float(norm) - want) < 1e-6 * want
        assert abs(float(g[1][5]) - scale / max(1.0, want)) < 1e-6 * scale


@pytest.mark.gpu
def test_two_graphs_and_two_streams_at_once():
    """Two captured calls with workspaces of their own, replayed on two streams,
    and eager calls beside them."""
    dev = require_gpu()
    sets = [inputs(dev, n, n) for n in (6, 60)]
    want = [chain(d) for d in sets]
    graphs, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for d in sets:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(chain(d))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = chain(sets[1])
    torch.cuda.synchronize()
    for got, w in zip(outs + [eager], want + [want[1]]):
        assert all(same(a, b) for a, b in zip(got, w))


@pytest.mark.gpu
def test_named_streams_and_threads():
    dev = require_gpu()
    sets = [inputs(dev, n, n) for n in (1, 9, 33, 100)]
    want = [chain(d) for d in sets]
    torch.cuda.synchronize()
    got = [None] * len(sets)

    def work(i):
        s = torch.cuda.Stream(device=dev)
        for _ in range(5):
            got[i] = chain(sets[i], s)
        s.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert all(same(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


@pytest.mark.gpu
def test_along_the_wire():
    """A training step's gradient shards arrive in 8 bits, are reduced, clipped to
    a norm and applied; the new weights go out in MXFP8, and what arrives serves
    tokens through routing and the experts: against the same in 64 bits."""
    dev = require_gpu()
    g = torch.Generator(device=dev).manual_seed(3)
    w = {k: torch.randn(E, *s, generator=g, device=dev) * s[1] ** -0.5
         for k, s in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))}
    grads = []
    for v in w.values():
        shards = [fq.fp8q_quantize((torch.randn(v.numel(), generator=g, device=dev) * 1e-2).bfloat16(), fq.E4M3)
                  for _ in range(4)]
        grads.append(fq.fp8q_dequant_reduce([q for q, _ in shards], [s for _, s in shards], fq.E4M3))
    # as the all-gather half sends them: codes and scales, clipped by their scales
    coded = [fq.fp8q_quantize(t.bfloat16(), fq.E4M3) for t in grads]
    before = [fq.fp8q_dequantize(q, s, fq.E4M3).clone() for q, s in coded]
    for values, tensors, scales in ((grads, grads, None), (before, [q for q, _ in coded], [s for _, s in coded])):
        exact = sum(float(t.double().square().sum()) for t in values)
        sumsq = fq.fp8q_grad_sumsq(tensors, scales=scales)
        assert abs(float(sumsq) - exact) < 1e-12 * exact
        keep = [t.clone() for t in values]
        norm = fq.fp8q_grad_clip(tensors, sumsq, 1.0, scales=scales)
        assert abs(float(norm) - math.sqrt(exact)) < 1e-6 * math.sqrt(exact)
        by = 1.0 / (math.sqrt(exact) + 1e-6)
        assert by < 0.5
        now = values if scales is None else [fq.fp8q_dequantize(q, s, fq.E4M3) for q, s in coded]
        for a, b in zip(now, keep):        # the factor, a scale and a value rounded
            assert float((a.double() - b.double() * by).abs().max()) <= 3 * ref.U32 * float(b.abs().max()) * by
    received = {}
    for (k, v), d in zip(w.items(), grads):
        v -= d.view(v.shape)
        received[k] = fq.mx8_quantize(v.bfloat16())
    x = torch.randn(3, H, generator=g, device=dev).bfloat16()
    weights, ids = fq.fp8q_moe_route(torch.randn(3, E, generator=g, device=dev), K)
    y = fq.fp8q_moe_experts(x, ids, weights, *[q for q, _ in received.values()],
                            **{k + "_scales": s for k, (_, s) in received.items()})
    values = [fq.mx8_dequantize(q, s).view(w[k].shape).double().cpu().numpy() for k, (q, s) in received.items()]
    want, bound = ref.experts(x.double().cpu().numpy(), ids.cpu().numpy(), weights.cpu().numpy(), *values, True)
    assert (abs(y.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.gpu
def test_few_tokens_equal_the_sorted_way():
    """The same experts by sort, permute, products in 64 bits and combine."""
    dev = require_gpu()
    d = inputs(dev, 12, 5)
    weights, ids = fq.fp8q_moe_route(d["logits"], K)
    y = fq.fp8q_moe_experts(d["x"], ids, weights, d["gate"], d["up"], d["down"], gate_scales=d["gate_scales"],
                            up_scales=d["up_scales"], down_scales=d["down_scales"]).double()
    slots, pairs, offsets = fq.fp8q_moe_sort(ids, E)
    rows, _ = fq.fp8q_moe_permute(d["x"], slots)
    m = {k: fq.mx8_dequantize(d[k], d[k + "_scales"]).view(d[k].shape).double() for k in ("gate", "up", "down")}
    ends, parts = offsets.tolist(), []
    for e in range(E):
        r = rows[ends[e]:ends[e + 1]].double()
        parts.append((torch.nn.functional.silu(r @ m["gate"][e].T) * (r @ m["up"][e].T)) @ m["down"][e].T)
    want = fq.fp8q_moe_combine(torch.cat(parts).bfloat16(), slots, weights, out_dtype=torch.float32).double()
    # both round to bf16 once: the rows there, the sum here
    assert float((y - want).abs().max()) <= 4 * 2.0 ** -8 * float(want.abs().max())


SMALL_GRID = os.path.join(HERE, "native", "libfp8q_model_small_grid.so")


@pytest.mark.gpu
def test_grids_that_have_to_be_split():
    """A build with grids of at most 64 waves: routing in several launches, and
    clipping whose workgroups take several chunks."""
    dev = require_gpu()
    if not os.path.exists(SMALL_GRID):
        pytest.skip("the small-grid build is missing: __graft_entry__.build() makes it")
    L = model.model_lib(SMALL_GRID)
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for tokens, experts, topk in ((1000, 128, 8), (300, 512, 6)):
        l = torch.randn(tokens, experts, device=dev)
        w, ids = torch.full((tokens + 1, topk), 9.0, device=dev), torch.full((tokens + 1, topk), 9, dtype=torch.int32, device=dev)
        assert L.fp8q_moe_route(l.data_ptr(), 0, tokens, experts, topk, 1, w.data_ptr(), ids.data_ptr(), st) == 0
        want = fq.fp8q_moe_route(l, topk)
        assert torch.equal(w[:-1], want[0]) and torch.equal(ids[:-1], want[1]) and (w[-1] == 9).all()
        dw, d = torch.randn(tokens, topk, device=dev), torch.empty_like(l)
        for norm in (0, 1):
            assert L.fp8q_moe_route_backward(dw.data_ptr(), l.data_ptr(), 0, w.data_ptr(), ids.data_ptr(), tokens,
                                             experts, topk, norm, d.data_ptr(), st) == 0
            assert torch.equal(d, fq.fp8q_moe_route_backward(dw, l, w[:-1], ids[:-1], normalize=bool(norm)))
    t = torch.randn(1 << 20, device=dev)
    norm, s = torch.zeros(1, device=dev), torch.tensor([16.0], dtype=torch.float64, device=dev)
    g = (model.Grad * 1)(model.Grad(t.data_ptr(), None, t.numel(), 0, 0))
    want = t * 0.25
    assert L.fp8q_grad_clip(g, 1, s.data_ptr(), 1.0, 0.0, norm.data_ptr(), st) == 0
    assert torch.equal(t, want) and float(norm) == 4.0


# On which stream a call allocates (no GPU).

CALLS = [("moe_route", 2, lambda t, s: fq.fp8q_moe_route(t[0], 4, weights_out=t[1], stream=s), 2),
         ("moe_route_backward", 1, lambda t, s: fq.fp8q_moe_route_backward(*t[:4], stream=s), 4),
         ("moe_experts", 1, lambda t, s: fq.fp8q_moe_experts(*t[:6], gate_scales=t[6], up_scales=t[7],
                                                             down_scales=t[8], workspace=t[9], stream=s), 10),
         ("grad_sumsq", 1, lambda t, s: fq.fp8q_grad_sumsq(t[:2], scales=[None, t[2]], workspace=t[3], stream=s), 4),
         ("grad_clip", 1, lambda t, s: fq.fp8q_grad_clip((t[0], t[1]), t[2], 1.0, scales=[t[3], None], stream=s), 4)]


@pytest.mark.parametrize("name,outputs,call,count", CALLS)
@pytest.mark.parametrize("named", [True, False])
def test_the_stream_of_allocations_and_records(monkeypatch, name, outputs, call, count, named):
    streams = FakeStreams(monkeypatch)
    made, seen = [], []

    class Binding:
        @staticmethod
        def function(*args):
            seen.append((streams.now.name, args[-1]))
            made[:] = [logged(4) for _ in range(outputs)]
            return (0, *made)

    setattr(Binding, name, Binding.function)
    monkeypatch.setattr(model, "_native", Binding)
    tensors = [logged(4) for _ in range(count)]
    call(tensors, streams.named if named else None)
    assert streams.now is streams.caller
    if named:
        assert seen == [("named", 2)]
        assert all("named" in recorded(t) for t in tensors)
        assert all("caller" in recorded(t) for t in made)
    else:
        assert seen == [("caller", 1)] and not any(recorded(t) for t in [*tensors, *made])
