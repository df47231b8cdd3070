"""Where a layer operator's call on a named stream allocates: from that
stream's memory.  A block that the current stream released with work on it still
pending must not become an output or a workspace that the named stream writes
at the same time.  Here (no GPU) a binding that allocates nothing says which
stream is current while it would; on a GPU the allocator's own segments do."""
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
from dequantize_reduce_transfer_amd import layer
from gpu_util import require_gpu
from stream_fakes import FakeStreams, logged, recorded

CALLS = [("rms_norm_quantize", 5, lambda t, s: fq.fp8q_rms_norm_quantize(t[0], t[1], residual=t[2], stream=s), 3),
         ("rms_norm_quantize", 5, lambda t, s: fq.mx8_rms_norm_quantize(t[0], t[1], h_out=t[2], stream=s), 3),
         ("rms_norm_backward", 2, lambda t, s: fq.fp8q_rms_norm_backward(*t[:4], dh=t[4], workspace=t[5], stream=s), 6),
         ("moe_sort", 3, lambda t, s: fq.fp8q_moe_sort(t[0], 8, workspace=t[1], stream=s), 2),
         ("moe_permute", 2, lambda t, s: fq.fp8q_moe_permute(t[0], t[1], scales=t[2], stream=s), 3),
         ("moe_combine", 1, lambda t, s: fq.fp8q_moe_combine(*t[:3], scales=t[3], stream=s), 4),
         ("moe_combine_backward", 2, lambda t, s: fq.fp8q_moe_combine_backward(*t[:4], stream=s), 4)]


@pytest.mark.parametrize("name,outputs,call,inputs", CALLS)
def test_a_named_stream_is_current_while_the_binding_allocates(monkeypatch, name, outputs, call, inputs):
    streams = FakeStreams(monkeypatch)
    made, seen = [], []

    class Binding:
        @staticmethod
        def function(*args):
            seen.append((streams.now.name, args[-1]))
            made[:] = [logged(4) for _ in range(outputs)]
            return (0, *made)

    setattr(Binding, name, Binding.function)
    monkeypatch.setattr(layer, "_native", Binding)
    tensors = [logged(4) for _ in range(inputs)]
    call(tensors, streams.named)
    assert seen == [("named", 2)] and streams.now is streams.caller
    assert all("named" in recorded(t) for t in tensors)          # memory of another stream's, maybe
    assert all("caller" in recorded(t) for t in made)            # which will read and release them


@pytest.mark.parametrize("name,outputs,call,inputs", CALLS)
def test_a_call_on_the_current_stream_records_nothing(monkeypatch, name, outputs, call, inputs):
    streams = FakeStreams(monkeypatch)
    made, seen = [], []

    class Binding:
        @staticmethod
        def function(*args):
            seen.append(streams.now.name)
            made[:] = [logged(4) for _ in range(outputs)]
            return (0, *made)

    setattr(Binding, name, Binding.function)
    monkeypatch.setattr(layer, "_native", Binding)
    monkeypatch.setattr(layer, "_raw_stream", lambda device: 1)
    tensors = [logged(4) for _ in range(inputs)]
    call(tensors, None)
    assert seen == ["caller"] and not any(recorded(t) for t in [*tensors, *made])


def test_a_refused_call_leaves_its_stream(monkeypatch):
    streams = FakeStreams(monkeypatch)

    class Binding:
        @staticmethod
        def moe_sort(*args):
            return (2, None, None, None)

    monkeypatch.setattr(layer, "_native", Binding)
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_moe_sort(logged(4), 8, stream=streams.named)
    assert streams.now is streams.caller


def _stream_of(t):
    """The raw handle of the stream that the tensor's memory belongs to."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not memory of the allocator's")


def _inputs(dev, tokens, hidden=768, topk=8, experts=64):
    g = torch.Generator(device=dev).manual_seed(tokens)

    def bf(*shape):
        return torch.randn(*shape, generator=g, device=dev).bfloat16()

    return dict(x=bf(tokens, hidden), w=torch.rand(hidden, generator=g, device=dev), dy=bf(tokens, hidden),
                ids=torch.rand(tokens, experts, generator=g, device=dev).topk(topk, 1).indices,
                rows=bf(tokens * topk, hidden), p=torch.rand(tokens, topk, generator=g, device=dev))


def _chain(d, stream):
    n = fq.fp8q_rms_norm_quantize(d["x"], d["w"], residual=d["dy"], want_y=True, want_rstd=True, stream=stream)
    m = fq.mx8_rms_norm_quantize(d["x"], d["w"], stream=stream)
    slots, pairs, offsets = fq.fp8q_moe_sort(d["ids"], 64, stream=stream)
    rows, scales = fq.fp8q_moe_permute(n.q, slots, scales=n.scales, stream=stream)
    y = fq.fp8q_moe_combine(d["rows"], slots, d["p"], stream=stream)
    drows, dp = fq.fp8q_moe_combine_backward(d["dy"], d["rows"], slots, d["p"], stream=stream)
    dx, dw = fq.fp8q_rms_norm_backward(y, n.h, d["w"], n.rstd, stream=stream)
    return [*n, m.q, m.scales, slots, pairs, offsets, rows, scales, y, drows, dp, dx, dw]


@pytest.mark.gpu
def test_outputs_are_the_named_streams_memory():
    dev = require_gpu()
    d = _inputs(dev, 700)
    current = [_stream_of(t) for t in _chain(d, None)]
    torch.cuda.synchronize()
    st = torch.cuda.Stream(device=dev)
    out = _chain(d, st)
    st.synchronize()
    assert set(current) == {torch.cuda.current_stream(dev).cuda_stream}
    assert {_stream_of(t) for t in out} == {st.cuda_stream}


@pytest.mark.gpu
def test_memory_with_work_pending_is_not_taken():
    """The current stream has a millisecond of work ahead of writes into blocks
    that are released at once; a chain on another stream whose inputs are ready,
    and which waits for nothing, keeps its results, its workspaces' included."""
    dev = require_gpu()
    d = _inputs(dev, 3000)
    want = [t.clone() for t in _chain(d, None)]
    sizes = [t.numel() * t.element_size() for t in want]
    sizes += [fq.fp8q_moe_sort_workspace(3000, 8, 64), fq.fp8q_rms_norm_backward_workspace(3000, 768)]
    busy = torch.empty(1 << 28, dtype=torch.bfloat16, device=dev)
    st = torch.cuda.Stream(device=dev)
    torch.cuda.synchronize()
    for _ in range(4):
        for _ in range(10):
            busy.fill_(1.0)
        for _ in range(3):
            for n in sizes:
                torch.empty(n, dtype=torch.uint8, device=dev).fill_(0xEE)      # released here
        got = _chain(d, st)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        del got
