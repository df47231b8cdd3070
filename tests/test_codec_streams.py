"""Where a codec call on a named stream allocates its outputs: from that
stream's memory, and not from blocks that the current stream released with work
on them still pending."""
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
from gpu_util import require_gpu
from stream_fakes import FakeStreams, logged, recorded

BF, U8, F32 = torch.bfloat16, torch.uint8, torch.float32
N = 4096


def shard():
    return dict(x=logged(N, dtype=BF), q=logged(N), s=logged(N // 128, dtype=F32), y=logged(N, dtype=F32),
                e=logged(N // 32))


CALLS = {
    "quantize": lambda d, s: fq.fp8q_quantize(d["x"], stream=s),
    "dequantize": lambda d, s: fq.fp8q_dequantize(d["q"], d["s"], stream=s),
    "reduce": lambda d, s: fq.fp8q_dequant_reduce([d["q"]], [d["s"]], stream=s),
    "requantize": lambda d, s: fq.fp8q_dequant_reduce_requantize([d["q"]], [d["s"]], stream=s),
    "sum": lambda d, s: fq.fp8q_sum_f32([d["y"]], stream=s),
    "mx8_quantize": lambda d, s: fq.mx8_quantize(d["x"], stream=s),
    "mx8_dequantize": lambda d, s: fq.mx8_dequantize(d["q"], d["e"], stream=s),
    "mx8_reduce": lambda d, s: fq.mx8_dequant_reduce([d["q"]], [d["e"]], stream=s),
    "tensorwise": lambda d, s: fq.fp8q_quantize_tensorwise(d["x"], stream=s),
}


class Library:
    """Every entry point succeeds and does nothing."""

    def __getattr__(self, name):
        return lambda *args: 0


@pytest.mark.parametrize("call", CALLS, ids=str)
def test_a_named_stream_is_current_while_outputs_are_allocated(monkeypatch, call):
    streams = FakeStreams(monkeypatch)
    monkeypatch.setattr(fq, "lib", Library)
    d = shard()
    made = []

    def empty(shape, dtype, device):
        made.append((logged(shape, dtype=dtype), streams.now.name))
        return made[-1][0]

    monkeypatch.setattr(torch, "empty", empty)
    CALLS[call](d, streams.named)
    assert made and all(on == "named" for _, on in made) and streams.now is streams.caller
    assert all(recorded(t) == {"named", "caller"} for t, _ in made)
    assert any("named" in recorded(t) for t in d.values())
    made.clear()
    CALLS[call](d, None)
    assert made and all(on == "caller" and not recorded(t) for t, on in made)


def _stream_of(t):
    """The raw handle of the stream that the tensor's memory belongs to."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not memory of the allocator's")


@pytest.mark.gpu
def test_outputs_are_the_named_streams_memory():
    dev = require_gpu()
    x = torch.randn(1 << 20, device=dev).bfloat16()
    torch.cuda.synchronize()
    st = torch.cuda.Stream(device=dev)
    q, s = fq.fp8q_quantize(x, stream=st)
    mq, e = fq.mx8_quantize(x, stream=st)
    out = [q, s, mq, e, *fq.fp8q_quantize_tensorwise(x, stream=st), fq.fp8q_dequantize(q, s, stream=st),
           fq.mx8_dequantize(mq, e, stream=st), fq.fp8q_dequant_reduce([q, q], [s, s], stream=st)]
    st.synchronize()
    assert {_stream_of(t) for t in out} == {st.cuda_stream}


@pytest.mark.gpu
def test_memory_with_work_pending_is_not_taken():
    """The current stream has a millisecond of work ahead of writes into blocks
    that are released at once; a quantize on another stream, whose input is
    ready and which waits for nothing, keeps its outputs."""
    dev = require_gpu()
    x = torch.randn(1 << 22, device=dev).bfloat16()
    want = [t.clone() for t in fq.fp8q_quantize(x)]
    busy = torch.empty(1 << 28, dtype=torch.bfloat16, device=dev)
    st = torch.cuda.Stream(device=dev)
    torch.cuda.synchronize()
    for _ in range(4):
        for _ in range(10):
            busy.fill_(1.0)
        for _ in range(3):
            for t in want:
                torch.empty_like(t).view(torch.uint8).fill_(0xEE)              # released here
        got = fq.fp8q_quantize(x, stream=st)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
        del got
