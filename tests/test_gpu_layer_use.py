"""The layer operators as a program uses them: captured in a HIP graph, on
named streams, from several threads, with offsets past 32 bits, in grids that
have to be split, with arguments that do not fit, and together in the example's
layer."""
import ctypes
import os
import sys
import threading

import numpy as np
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
from dequantize_reduce_transfer_amd import layer
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
EPS = 1e-6


def same(a, b):
    return (a is None and b is None) or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def inputs(dev, tokens=300, hidden=544, topk=4, experts=24, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)

    ids = torch.rand(tokens, experts, generator=g, device=dev).topk(topk, 1).indices
    return dict(x=bf(tokens, hidden), res=bf(tokens, hidden), w=torch.rand(hidden, generator=g, device=dev),
                ids=ids, experts=experts, dy=bf(tokens, hidden), expert_out=bf(tokens * topk, hidden),
                weights=torch.rand(tokens, topk, generator=g, device=dev))


def chain(d, stream=None):
    """Every entry point once, each on what the one before it made."""
    kw = dict(stream=stream)
    n8 = fq.fp8q_rms_norm_quantize(d["x"], d["w"], EPS, residual=d["res"], want_y=True, want_rstd=True, **kw)
    mx = fq.mx8_rms_norm_quantize(d["x"], d["w"], EPS, residual=d["res"], want_rstd=True, **kw)
    slots, pairs, offsets = fq.fp8q_moe_sort(d["ids"], d["experts"], **kw)
    rows, scales = fq.fp8q_moe_permute(n8.q, slots, scales=n8.scales, **kw)
    mrows, mscales = fq.fp8q_moe_permute(mx.q, slots, scales=mx.scales, **kw)
    y8 = fq.fp8q_moe_combine(rows, slots, d["weights"], scales=scales, out_dtype=torch.float32, **kw)
    ym = fq.fp8q_moe_combine(mrows, slots, d["weights"], scales=mscales, **kw)
    yb = fq.fp8q_moe_combine(d["expert_out"], slots, d["weights"], **kw)
    drows, dw = fq.fp8q_moe_combine_backward(d["dy"], d["expert_out"], slots, d["weights"], **kw)
    dx, dweight = fq.fp8q_rms_norm_backward(yb, n8.h, d["w"], n8.rstd, dh=d["dy"], **kw)
    return [*n8, *mx, slots, pairs, offsets, rows, scales, mrows, mscales, y8, ym, yb, drows, dw, dx, dweight]


def test_graph_replays_equal_eager():
    dev = require_gpu()
    for tokens in (3, 300, 3000):           # one workgroup of each size, and two kernels, sort them
        d = inputs(dev, tokens=tokens, seed=tokens)
        want = [t if t is None else t.clone() for t in chain(d)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            chain(d)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = chain(d)
        for _ in range(4):
            for t in outs:
                if t is not None:
                    t.view(torch.uint8).fill_(0xA5)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(outs, want))


def test_named_stream_and_released_tensors():
    """A chain on a named stream while the current stream allocates and writes
    memory; intermediates are released before the stream has read them."""
    dev = require_gpu()
    d = inputs(dev, tokens=4000, hidden=1024)
    want = chain(d)
    torch.cuda.synchronize()
    st = torch.cuda.Stream(device=dev)
    st.wait_stream(torch.cuda.current_stream(dev))
    busy = torch.empty(1 << 28, dtype=torch.bfloat16, device=dev).fill_(1.0)
    torch.cuda.synchronize()
    for _ in range(10):                     # a few ms of work ahead of the chain
        fq.fp8q_quantize(busy, fq.E4M3, stream=st)
    got = chain(d, stream=st)
    keep = [4, 12, 17, 19, 20, 21, 22, 23]  # the rest is released here
    got = {i: got[i] for i in keep}
    junk = [torch.full((4000 * 1024,), 7, dtype=torch.bfloat16, device=dev) for _ in range(24)]
    st.synchronize()
    torch.cuda.synchronize()
    assert all(same(got[i], want[i]) for i in keep)
    del junk, busy


def test_threads_on_their_own_streams():
    dev = require_gpu()
    jobs = [inputs(dev, tokens=500 + 700 * j, seed=j) for j in range(4)]
    want = [chain(d) for d in jobs]
    torch.cuda.synchronize()
    got, errors = [None] * 4, []

    def work(i):
        try:
            st = torch.cuda.Stream(device=dev)
            with torch.cuda.stream(st):
                for _ in range(10):
                    got[i] = chain(jobs[i])
                st.synchronize()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(same(x, y) for x, y in zip(a, b))


def test_offsets_past_32_bits():
    """Rows whose elements (norm, combine) and bytes (permute) lie past 2^32:
    the last rows equal the same rows alone."""
    dev = require_gpu()
    hidden, rows = 2048, (1 << 21) + 1030           # 2^32 + 2109440 elements
    x = torch.randn(1024, hidden, device=dev).to(torch.bfloat16).repeat(rows // 1024 + 1, 1)[:rows].contiguous()
    w = torch.rand(hidden, device=dev)
    last = x[-1030:].clone()
    out = fq.fp8q_rms_norm_quantize(x, w, EPS, want_rstd=True)
    alone = fq.fp8q_rms_norm_quantize(last, w, EPS, want_rstd=True)
    torch.cuda.synchronize()
    assert same(out.q[-1030:].clone(), alone.q) and same(out.scales[-1030:].clone(), alone.scales)
    assert same(out.rstd[-1030:].clone(), alone.rstd) and same(out.q[:1024].clone(), out.q[1024:2048].clone())
    dx, _ = fq.fp8q_rms_norm_backward(x, x, w, out.rstd)
    dx1, _ = fq.fp8q_rms_norm_backward(last, last, w, alone.rstd)
    torch.cuda.synchronize()
    assert same(dx[-1030:].clone(), dx1)
    del dx
    slots = torch.arange(rows - 1, rows - 1 - 64, -1, dtype=torch.int32, device=dev).reshape(16, 4)
    big = fq.fp8q_moe_permute(out.q[:16].contiguous(), slots, scales=out.scales[:16].contiguous(),
                              out=torch.zeros_like(out.q), scales_out=torch.zeros_like(out.scales))
    torch.cuda.synchronize()
    for t in range(16):
        for j in range(4):
            at = rows - 1 - (4 * t + j)
            assert same(big[0][at], out.q[t]) and same(big[1][at], out.scales[t])
    weights = torch.rand(16, 4, device=dev)
    y = fq.fp8q_moe_combine(x, slots, weights)
    near = slots - (rows - 1030)
    y1 = fq.fp8q_moe_combine(last, near, weights)
    y8 = fq.fp8q_moe_combine(big[0], slots, weights, scales=big[1])
    y81 = fq.fp8q_moe_combine(big[0][-1030:].contiguous(), near, weights, scales=big[1][-1030:].contiguous())
    dy = torch.randn(16, hidden, device=dev).to(torch.bfloat16)
    drows, dw = fq.fp8q_moe_combine_backward(dy, x, slots, weights, drows_out=torch.zeros_like(x))
    drows1, dw1 = fq.fp8q_moe_combine_backward(dy, last, near, weights, drows_out=torch.zeros_like(last))
    torch.cuda.synchronize()
    assert same(y, y1) and same(y8, y81) and same(dw, dw1)
    assert same(drows[-1030:].clone(), drows1) and not drows[:-1030].any()


SMALL = os.path.join(HERE, "native", "libfp8q_layer_small_grid.so")


@pytest.mark.parametrize("rows,hidden", [(100, 72), (333, 1030), (37, 8192), (9, 20000), (521, 16392)])
@pytest.mark.parametrize("in_place", [None, "dy", "dh"])
def test_split_norm_gradients_equal_whole_ones(rows, hidden, in_place):
    dev = require_gpu()
    if not os.path.exists(SMALL):
        pytest.skip("the small-grid library is built by __graft_entry__.build()")
    S = layer.layer_lib(SMALL)
    g = torch.Generator(device=dev).manual_seed(rows * hidden)
    dy, h, dh = (torch.randn(rows, hidden, generator=g, device=dev).bfloat16() for _ in range(3))
    w = torch.rand(hidden, generator=g, device=dev)
    rstd = torch.rand(rows, generator=g, device=dev) + 0.5
    ws = torch.empty(fq.fp8q_rms_norm_backward_workspace(rows, hidden), dtype=torch.uint8, device=dev)
    out = []
    for lib in (layer.layer_lib(), S):
        d = dict(dy=dy.clone(), dh=dh.clone())
        dx = d[in_place] if in_place else torch.zeros_like(h)
        dw = torch.zeros(hidden, device=dev)
        torch.cuda.synchronize()
        P = ctypes.c_void_p
        assert lib.fp8q_rms_norm_backward(P(d["dy"].data_ptr()), P(h.data_ptr()), P(w.data_ptr()), 0,
                                          P(rstd.data_ptr()), P(d["dh"].data_ptr()), rows, hidden, P(dx.data_ptr()),
                                          P(dw.data_ptr()), P(ws.data_ptr() or None), ws.numel(), None) == 0
        torch.cuda.synchronize()
        out.append((dx, dw))
    assert same(out[0][0], out[1][0]) and same(out[0][1], out[1][1])


def test_split_launches_equal_whole_ones():
    """A build whose grids hold 64 waves splits every launch here; its outputs
    equal the library's bit for bit."""
    dev = require_gpu()
    if not os.path.exists(SMALL):
        pytest.skip("the small-grid library is built by __graft_entry__.build()")
    S = layer.layer_lib(SMALL)
    P = ctypes.c_void_p

    def p(t):
        return P(t.data_ptr()) if t is not None else None

    for hidden in (72, 512, 1030, 2048):
        d = inputs(dev, tokens=333, hidden=hidden, topk=9, experts=20, seed=hidden)
        rows = 333
        want = fq.fp8q_rms_norm_quantize(d["x"], d["w"], EPS, residual=d["res"], want_y=True, want_rstd=True)
        got = [torch.full_like(t, 0x5A if t.dtype == torch.uint8 else 7) for t in want]
        torch.cuda.synchronize()
        assert S.fp8q_rms_norm_quantize(p(d["x"]), p(d["res"]), p(d["w"]), 0, EPS, rows, hidden, 0, p(got[2]),
                                        p(got[3]), p(got[0]), p(got[1]), p(got[4]), None) == 0
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
        if hidden % 32 == 0:
            want = fq.mx8_rms_norm_quantize(d["x"], d["w"], EPS, residual=d["res"], want_y=True, want_rstd=True)
            got = [torch.full_like(t, 0x5A if t.dtype == torch.uint8 else 7) for t in want]
            torch.cuda.synchronize()
            assert S.mx8_rms_norm_quantize(p(d["x"]), p(d["res"]), p(d["w"]), 0, EPS, rows, hidden, p(got[2]),
                                           p(got[3]), p(got[0]), p(got[1]), p(got[4]), None) == 0
            torch.cuda.synchronize()
            assert all(same(a, b) for a, b in zip(got, want))
        slots, _, _ = fq.fp8q_moe_sort(d["ids"], 20)
        n8 = fq.fp8q_rms_norm_quantize(d["x"], d["w"], EPS)
        wr, ws = fq.fp8q_moe_permute(n8.q, slots, scales=n8.scales)
        gr, gs = torch.zeros_like(wr), torch.zeros_like(ws)
        torch.cuda.synchronize()
        assert S.fp8q_moe_permute(p(n8.q), hidden, p(n8.scales), 4 * n8.scales.shape[1], p(slots), 333, 9,
                                  333 * 9, p(gr), p(gs), None) == 0
        torch.cuda.synchronize()
        assert same(gr, wr) and same(gs, ws)
        for f, (r, s) in ((0, (d["expert_out"], None)), (1, (wr, ws))):
            for od, dt in ((0, torch.float32), (1, torch.bfloat16)):
                want = fq.fp8q_moe_combine(r, slots, d["weights"], scales=s, out_dtype=dt)
                got = torch.zeros_like(want)
                torch.cuda.synchronize()
                assert S.fp8q_moe_combine(p(r), f, p(s), p(slots), p(d["weights"]), 333, 9, 333 * 9, hidden,
                                          p(got), od, None) == 0
                torch.cuda.synchronize()
                assert same(got, want)
        want = fq.fp8q_moe_combine_backward(d["dy"], d["expert_out"], slots, d["weights"])
        got = [torch.zeros_like(t) for t in want]
        torch.cuda.synchronize()
        assert S.fp8q_moe_combine_backward(p(d["dy"]), p(d["expert_out"]), p(slots), p(d["weights"]), 333, 9,
                                           333 * 9, hidden, p(got[0]), p(got[1]), None) == 0
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))


def test_refusals():
    dev = require_gpu()
    bf = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    f32, i32 = torch.zeros(4, 64, device=dev), torch.zeros(4, 2, dtype=torch.int32, device=dev)
    u8 = torch.zeros(8, 64, dtype=torch.uint8, device=dev)
    w, rstd, w2 = torch.ones(64, device=dev), torch.ones(4, device=dev), torch.ones(4, 2, device=dev)
    bad_values = [
        lambda: fq.fp8q_rms_norm_quantize(bf, w[:32]),
        lambda: fq.fp8q_rms_norm_quantize(bf, w, fmt=2),
        lambda: fq.fp8q_rms_norm_quantize(bf, w, residual=bf[:3]),
        lambda: fq.fp8q_rms_norm_quantize(bf, w, h_out=torch.empty_like(bf)),
        lambda: fq.fp8q_rms_norm_quantize(bf.t(), torch.ones(4, device=dev)),
        lambda: fq.fp8q_rms_norm_quantize(bf, w, q_out=u8),
        lambda: fq.fp8q_rms_norm_quantize(bf, w.cpu()),
        lambda: fq.mx8_rms_norm_quantize(bf[:, :40].contiguous(), w[:40]),
        lambda: fq.fp8q_rms_norm_backward(bf, bf[:3], w, rstd[:3]),
        lambda: fq.fp8q_rms_norm_backward(bf, bf, w, rstd[:3]),
        lambda: fq.fp8q_rms_norm_backward(bf, bf, w, rstd, dh=bf[:2]),
        lambda: fq.fp8q_moe_sort(i32.reshape(-1), 4),
        lambda: fq.fp8q_moe_sort(i32, 0),
        lambda: fq.fp8q_moe_sort(i32, 1025),
        lambda: fq.fp8q_moe_sort(torch.zeros(2, 65, dtype=torch.int32, device=dev), 8),
        lambda: fq.fp8q_moe_permute(bf, i32[:3]),
        lambda: fq.fp8q_moe_permute(bf, i32, out=torch.empty(8, 32, dtype=torch.bfloat16, device=dev)),
        lambda: fq.fp8q_moe_permute(bf, i32, scales_out=f32),
        lambda: fq.fp8q_moe_combine(bf, i32, w2[:2]),
        lambda: fq.fp8q_moe_combine(bf, i32, scales=f32),
        lambda: fq.fp8q_moe_combine(u8, i32, scales=f32),
        lambda: fq.fp8q_moe_combine(u8, i32, scales=torch.zeros(8, 1, device=dev), fmt=7),
        lambda: fq.fp8q_moe_combine_backward(bf, bf[:, :32].contiguous(), i32, w2),
        lambda: fq.fp8q_moe_combine_backward(bf, bf, i32, w2[:1]),
    ]
    for i, call in enumerate(bad_values):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was taken" % i)
    for i, call in enumerate([
            lambda: fq.fp8q_rms_norm_quantize(f32, w),
            lambda: fq.fp8q_rms_norm_quantize(bf, w.double()),
            lambda: fq.fp8q_rms_norm_quantize(bf, w, q_out=bf),
            lambda: fq.fp8q_rms_norm_quantize(bf, w, "small"),
            lambda: fq.fp8q_moe_sort(f32, 4),
            lambda: fq.fp8q_moe_permute(bf, i32.long()),
            lambda: fq.fp8q_moe_permute(bf, i32, out=torch.empty(8, 64, device=dev)),
            lambda: fq.fp8q_moe_combine(u8, i32),
            lambda: fq.fp8q_moe_combine(u8, i32, scales=bf),
            lambda: fq.fp8q_moe_combine_backward(f32, bf, i32, w2)]):
        with pytest.raises(TypeError):
            call()
            pytest.fail("call %d was taken" % i)
    for call in (lambda: fq.fp8q_rms_norm_quantize(bf, w, float("nan")),
                 lambda: fq.fp8q_rms_norm_quantize(bf, w, -1.0),
                 lambda: fq.fp8q_rms_norm_quantize(torch.zeros(1, 32800, dtype=torch.bfloat16, device=dev),
                                                   torch.ones(32800, device=dev)),
                 lambda: fq.fp8q_rms_norm_quantize(bf, w, residual=bf, y_out=bf)):
        with pytest.raises(fq.Fp8qError):
            call()


def test_memory_that_runs_out_raises_as_in_torch():
    """An output that this process's limit of 2 GiB cannot hold: the exception
    that torch's own allocations (and the codec's functions) raise, and the next
    call goes through."""
    dev = require_gpu()
    torch.cuda.empty_cache()
    x = torch.zeros(1 << 12, 1 << 14, dtype=torch.uint8, device=dev)
    slots = torch.full((1 << 12, 64), -1, dtype=torch.int32, device=dev)
    total = torch.cuda.get_device_properties(dev).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved(dev) + (2 << 30)) / total, dev)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            fq.fp8q_moe_permute(x, slots)              # 2^18 rows of 16 KiB: 4 GiB
        rows, _ = fq.fp8q_moe_permute(x[:8], slots[:8])
        torch.cuda.synchronize()
        assert rows.shape == (512, 1 << 14)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0, dev)


def test_unaligned_views_are_refused_and_strided_ones_too():
    dev = require_gpu()
    base = torch.zeros(4 * 64 + 8, dtype=torch.bfloat16, device=dev)
    w = torch.ones(64, device=dev)
    with pytest.raises(fq.Fp8qError, match="ALIGN"):
        fq.fp8q_rms_norm_quantize(base[1:257].view(4, 64), w)
    with pytest.raises(ValueError, match="contiguous"):
        fq.fp8q_rms_norm_quantize(torch.zeros(4, 128, dtype=torch.bfloat16, device=dev)[:, ::2], w)


def test_example_layer_learns_and_matches_a_plain_layer():
    """The example's layer against the same layer in plain torch (32 bits):
    output and gradients agree to what 8-bit rows and bf16 give, and a few
    steps lower the loss."""
    require_gpu()
    sys.path.insert(0, os.path.join(os.path.dirname(HERE), "examples"))
    import moe_layer

    losses = moe_layer.main(["--tokens", "200", "--steps", "4"])
    assert losses[-1] < losses[0] and np.isfinite(losses).all()

    torch.manual_seed(1)
    m = moe_layer.MoeLayer(hidden=128, experts=8, topk=2)
    x = torch.randn(60, 128, device="cuda").to(torch.bfloat16).requires_grad_()
    r = torch.randn(60, 128, device="cuda").to(torch.bfloat16).requires_grad_()
    dout, dh = torch.randn(60, 128, device="cuda"), torch.randn(60, 128, device="cuda")
    out, h = m(x, r)
    ((out.float() * dout).sum() + (h.float() * dh).sum()).backward()
    got = [out.detach().float(), x.grad.float(), r.grad.float(), m.norm.grad, m.router.grad,
           m.weights.grad.float()]

    x2, r2 = (t.detach().float().requires_grad_() for t in (x, r))
    norm, router, weights = (t.detach().float().requires_grad_() for t in (m.norm, m.router, m.weights))
    h2 = x2 + r2
    y2 = h2 * torch.rsqrt(h2.square().mean(1, keepdim=True) + m.eps) * norm
    p2 = torch.softmax(y2 @ router, dim=1)
    ids = torch.softmax(m_y(m, x, r) @ m.router, dim=1).topk(2, dim=1).indices   # the layer's own choices
    w2 = torch.gather(p2, 1, ids)
    out2 = sum(w2[:, j, None] * torch.stack([y2[t] @ weights[ids[t, j]] for t in range(60)]) for j in range(2))
    ((out2 * dout).sum() + (h2 * dh).sum()).backward()
    want = [out2.detach(), x2.grad, r2.grad, norm.grad, router.grad, weights.grad]
    # E4M3 rows round by up to 2^-4, about 2.5% in the root mean square; products
    # of 128 terms average it, bf16 adds under 1%: 6% in the norm
    for i, (a, b) in enumerate(zip(got, want)):
        assert float((a - b).norm() / b.norm()) < 0.06, i


def m_y(m, x, r):
    return fq.mx8_rms_norm_quantize(x.detach(), m.norm.detach(), m.eps, residual=r.detach(), want_y=True).y.float()
