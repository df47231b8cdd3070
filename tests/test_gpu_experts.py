"""A whole MoE layer for a few tokens on the GPU against 64 bits, within the
bounds that model_ref derives, and bit for bit where every sum is exact."""
import numpy as np
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
import model_ref as ref
import oracle
from gpu_util import host, require_gpu

pytestmark = pytest.mark.gpu

BF16, E4M3, E5M2, MX8 = ref.BF16, ref.E4M3, ref.E5M2, ref.MX8
FORMATS = [pytest.param(f, id=n) for f, n in ((BF16, "bf16"), (E4M3, "e4m3"), (E5M2, "e5m2"), (MX8, "mx8"))]


class Layer:
    """Matrices of one format, on the GPU and as 64-bit values."""

    def __init__(self, fmt, experts, hidden, inter, seed, fused=False):
        self.fmt, self.experts, self.hidden, self.inter = fmt, experts, hidden, inter
        rng = np.random.default_rng(seed)
        self.t, self.s, self.v = {}, {}, {}
        for name, rows, width in (("gate", inter, hidden), ("up", inter, hidden), ("down", hidden, inter)):
            self.t[name], self.s[name], self.v[name] = self.matrix(rng, experts, rows, width)
        if fused:                          # gate and up as halves of one tensor
            for d in (self.t, self.s):
                if d["gate"] is not None:
                    shape = (experts, inter, -1)
                    both = torch.cat([d["gate"].view(shape), d["up"].view(shape)], 1)
                    d["gate"], d["up"] = both[:, :inter], both[:, inter:]

    def matrix(self, rng, experts, rows, width):
        dev = require_gpu()
        shape = (experts, rows, width)
        if self.fmt == BF16:
            t = torch.from_numpy(rng.normal(size=shape).astype(np.float32) * max(1, width) ** -0.5).bfloat16()
            return t.to(dev), None, t.double().numpy()
        q = rng.integers(0, 256, size=(experts * rows, width), dtype=np.uint8)
        v = oracle.fp8_decode(q, 1 if self.fmt == E5M2 else 0)
        top = 57344.0 if self.fmt == E5M2 else 448.0
        q[~np.isfinite(v)] = 0
        if self.fmt == E5M2:               # no two values of a row over a million apart
            q[np.abs(oracle.fp8_decode(q, 1)) > 64.0] &= 0x3F
            top = 64.0
        block = 32 if self.fmt == MX8 else 128
        blocks = -(-width // block)
        size = 2.0 / (top * max(1, width) ** 0.5)
        if self.fmt == MX8:
            s = (np.round(np.log2(size)) + 127 + rng.integers(-2, 3, size=(experts * rows, blocks))).astype(np.uint8)
        else:
            s = (size * np.exp(rng.normal(size=(experts * rows, blocks)))).astype(np.float32)
        scale = np.ldexp(1.0, s.astype(np.int64) - 127) if self.fmt == MX8 else s.astype(np.float64)
        value = oracle.fp8_decode(q, 1 if self.fmt == E5M2 else 0).astype(np.float64)
        value = value * scale[:, np.arange(width) // block] if width else value
        return (torch.from_numpy(q.reshape(shape)).to(dev), torch.from_numpy(s).to(dev), value.reshape(shape))

    def __call__(self, x, ids, w, **k):
        return fq.fp8q_moe_experts(x, ids, w, self.t["gate"], self.t["up"], self.t["down"],
                                   gate_scales=self.s["gate"], up_scales=self.s["up"], down_scales=self.s["down"],
                                   fmt=fq.E5M2 if self.fmt == E5M2 else fq.E4M3, **k)

    def want(self, x, ids, w, bf16):
        return ref.experts(x.double().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), self.v["gate"], self.v["up"],
                           self.v["down"], bf16)


def tokens_of(tokens, topk, experts, hidden, seed, gone=0.0, wide=False):
    dev = require_gpu()
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, hidden, generator=g).bfloat16().to(dev)
    ids = torch.stack([torch.randperm(max(experts, topk), generator=g)[:topk] % experts for _ in range(tokens)]) \
        if tokens else torch.zeros(0, topk, dtype=torch.int64)
    if gone:
        ids[torch.rand(tokens, topk, generator=g) < gone] = -1
    w = torch.rand(tokens, topk, generator=g).to(dev)
    return x, (ids if wide else ids.int()).to(dev), w


def check(layer, x, ids, w, dtype=torch.bfloat16, **k):
    got = layer(x, ids, w, out_dtype=dtype, **k)
    assert got.dtype == dtype and got.shape == x.shape
    want, bound = layer.want(x, ids, w, dtype == torch.bfloat16)
    err = np.abs(got.double().cpu().numpy() - want)
    worst = (err - bound).max() if err.size else 0.0
    assert worst <= 0.0, "%.3g past its bound" % worst
    return got


# hidden and inter around chunks of 64, blocks of 32 and 128, tiles of 16 rows
SIZES = [(64, 64), (128, 32), (32, 16), (256, 96), (416, 224), (512, 544), (1088, 64), (64, 1088)]
ODD = [(1, 1), (7, 3), (15, 17), (63, 65), (100, 40), (129, 31), (191, 257), (1411, 100)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hidden,inter", SIZES)
def test_sizes(fmt, hidden, inter):
    if fmt == MX8 and inter % 32:
        inter = 32
    layer = Layer(fmt, 7, hidden, inter, hidden + inter)
    for dtype in (torch.bfloat16, torch.float32):
        check(layer, *tokens_of(1, 3, 7, hidden, 1), dtype)
        check(layer, *tokens_of(9, 2, 7, hidden, 2, gone=0.2), dtype)


@pytest.mark.parametrize("fmt", FORMATS[:3])
@pytest.mark.parametrize("hidden,inter", ODD)
def test_odd_sizes(fmt, hidden, inter):
    layer = Layer(fmt, 5, hidden, inter, hidden + inter)
    for dtype in (torch.bfloat16, torch.float32):
        check(layer, *tokens_of(1, 2, 5, hidden, 1), dtype)
        check(layer, *tokens_of(11, 3, 5, hidden, 2, gone=0.2), dtype)


# tokens, topk, experts: fewer pairs than experts and more, an expert's pairs
# around 16, 32, 48 and 64, and the most that there may be
COUNTS = [(1, 1, 1), (1, 8, 128), (2, 8, 16), (5, 8, 128), (16, 1, 1), (17, 1, 1), (31, 2, 2), (33, 1, 1), (49, 1, 1),
          (64, 2, 2), (65, 1, 1), (70, 3, 3), (8, 8, 64), (64, 8, 128), (128, 8, 40), (130, 1, 1), (16, 64, 100),
          (40, 4, 1000), (1024, 1, 3)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,topk,experts", COUNTS)
def test_counts(fmt, tokens, topk, experts):
    layer = Layer(fmt, experts, 96, 64, tokens + topk)
    x, ids, w = tokens_of(tokens, topk, experts, 96, tokens, wide=tokens % 2 == 0)
    got = check(layer, x, ids, w)
    check(layer, x, ids, w, torch.float32)
    assert all(torch.equal(layer(x, ids, w).view(torch.int16), got.view(torch.int16)) for _ in range(3))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens", [20, 100])
def test_long_rows_of_few_experts(fmt, tokens):
    """down's k's in several parts, the last of them ragged (MXFP8: by 32)."""
    layer = Layer(fmt, 2, 160, 2144 if fmt == MX8 else 2153, 8)
    x, ids, w = tokens_of(tokens, 2, 2, 160, tokens, gone=0.1)
    for dtype in (torch.bfloat16, torch.float32):
        got = check(layer, x, ids, w, dtype)
        assert torch.equal(layer(x, ids, w, out_dtype=dtype), got)


@pytest.mark.parametrize("fmt", FORMATS)
def test_exact_sums(fmt):
    """Small integers throughout, and gates above 32 (there exp(-g) is lost
    beside 1, and silu(g) is g): nothing is rounded, and the fp32 output is the
    integer itself."""
    dev = require_gpu()
    E, I, H, T, K = 6, 160, 192, 20, 3
    rng = np.random.default_rng(1)
    x = rng.integers(0, 2, size=(T, H)).astype(np.float32)
    x[:, 0] = 1.0
    m = {"gate": rng.integers(0, 2, size=(E, I, H)), "up": rng.integers(-1, 2, size=(E, I, H)),
         "down": rng.integers(-1, 2, size=(E, H, I))}
    m["gate"][:, :, 0] = 32
    for k in ("up", "down"):                # few ones, so that sums stay small
        m[k] *= rng.random(m[k].shape) < 0.06
    layer = Layer.__new__(Layer)
    layer.fmt, layer.t, layer.s = fmt, {}, {}
    for k, v in m.items():
        if fmt == BF16:
            layer.t[k], layer.s[k] = torch.from_numpy(v.astype(np.float32)).bfloat16().to(dev), None
            continue
        # stored as twice the value, with a scale of one half
        codes = oracle.fp8_encode((2 * v).astype(np.float32).ravel(), 1 if fmt == E5M2 else 0).reshape(v.shape)
        blocks = -(-v.shape[2] // (32 if fmt == MX8 else 128))
        s = np.full((v.shape[0] * v.shape[1], blocks), 126 if fmt == MX8 else 0.5,
                    np.uint8 if fmt == MX8 else np.float32)
        layer.t[k], layer.s[k] = torch.from_numpy(codes).to(dev), torch.from_numpy(s).to(dev)
    ids = np.stack([rng.permutation(E)[:K] for _ in range(T)])
    w = rng.integers(1, 4, size=(T, K)).astype(np.float32)
    g, u = np.einsum("eih,th->tei", m["gate"], x), np.einsum("eih,th->tei", m["up"], x)
    y = np.einsum("ehi,tei->teh", m["down"], g * u)
    want = sum(w[:, j, None] * y[np.arange(T), ids[:, j]] for j in range(K))
    assert np.abs(want).max() < 2 ** 24 and g.min() >= 32 and np.abs(g * u).max() < 2 ** 16
    args = (torch.from_numpy(x).bfloat16().to(dev), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev))
    assert np.array_equal(host(layer(*args, out_dtype=torch.float32)), want.astype(np.float32))
    got = layer(*args)
    assert torch.equal(got.cpu(), torch.from_numpy(want.astype(np.float32)).bfloat16())


@pytest.mark.parametrize("fmt", FORMATS)
def test_gate_and_up_as_halves_of_one_tensor(fmt):
    apart, one = Layer(fmt, 6, 128, 64, 3), Layer(fmt, 6, 128, 64, 3, fused=True)
    assert not one.t["gate"].is_contiguous()
    x, ids, w = tokens_of(7, 2, 6, 128, 4)
    assert torch.equal(check(one, x, ids, w), apart(x, ids, w))


def test_what_the_codec_quantizes():
    """Weights as mx8_quantize and fp8q_quantize leave them (flat scales), and
    what the receiver dequantizes."""
    dev = require_gpu()
    g = torch.Generator().manual_seed(0)
    E, I, H = 8, 128, 256
    w = {k: (torch.randn(E, *s, generator=g) * 0.06).bfloat16().to(dev)
         for k, s in (("gate", (I, H)), ("up", (I, H)), ("down", (H, I)))}
    x, ids, p = tokens_of(6, 2, E, H, 5)
    for mx in (True, False):
        layer = Layer.__new__(Layer)
        layer.fmt, layer.t, layer.s, layer.v = MX8 if mx else E4M3, {}, {}, {}
        for k, t in w.items():
            if mx:
                layer.t[k], layer.s[k] = fq.mx8_quantize(t)
                v = fq.mx8_dequantize(layer.t[k], layer.s[k])
            else:
                q, layer.s[k] = fq.fp8q_quantize(t.view(-1), fq.E4M3)
                layer.t[k], v = q.view(t.shape), fq.fp8q_dequantize(q, layer.s[k], fq.E4M3)
            layer.v[k] = v.view(t.shape).double().cpu().numpy()
        check(layer, x, ids, p)


@pytest.mark.parametrize("fmt", FORMATS)
def test_padding_foreign_and_repeated_experts(fmt):
    layer = Layer(fmt, 4, 96, 32, 9)
    x, ids, w = tokens_of(6, 4, 4, 96, 6)
    ids[0] = -1                             # a padding token
    ids[1] = torch.tensor([4, 2 ** 31 - 1, -2 ** 31, -1])
    ids[2] = 3                              # one expert, four times
    ids[3] = torch.tensor([1, 9, 1, -5])
    w[0, 0] = float("nan")                  # of choices that are none: not used
    w[1, 1] = float("inf")
    want_w = w.clone()
    want_w[:2] = 0.0
    for i in (ids, ids.long()):
        for dtype in (torch.bfloat16, torch.float32):
            got = layer(x, i, w, out_dtype=dtype)
            want, bound = layer.want(x, ids, want_w, dtype == torch.bfloat16)
            assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
            assert not got[:2].any()
    big = ids.long()
    big[1] = torch.tensor([2 ** 32, 2 ** 32 + 1, -2 ** 40, 2 ** 62])
    assert torch.equal(layer(x, big, w), layer(x, ids, w))
    none = torch.full_like(ids, -1)
    assert not layer(x, none, w).any()


@pytest.mark.parametrize("fmt", FORMATS)
def test_special_values_stay_with_their_tokens_and_rows(fmt):
    """An inf or NaN in x, a weight or a scale reaches the outputs that use it,
    and no others."""
    layer = Layer(fmt, 4, 256, 64, 12)
    x, ids, w = tokens_of(8, 1, 4, 256, 6)
    ids[:, 0] = torch.tensor([0, 0, 1, 1, 2, 2, 3, 3])
    clean = layer(x, ids, w)
    bad = x.clone()
    bad[3, 100] = float("nan")
    got = layer(bad, ids, w)
    assert got[3].isnan().all()
    keep = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(got[keep], clean[keep])
    if fmt == BF16:
        layer.t["down"][2, 77, 5] = float("nan")
    else:
        layer.t["down"][2, 77, 5] = 0x7F    # NaN in both
    got = layer(x, ids, w)
    assert got[4:6, 77].isnan().all()
    got[4:6, 77] = clean[4:6, 77]
    assert torch.equal(got, clean)
    if fmt == MX8:
        layer.s["gate"].view(4, 64, -1)[1, 63, 2] = 255
    elif fmt != BF16:
        layer.s["gate"].view(4, 64, -1)[1, 63, 1] = float("nan")
    else:
        layer.t["gate"][1, 63, 200] = float("inf")
    got = layer(x, ids, w)                  # silu(inf) is inf, silu(-inf) is NaN
    assert not got[2:4].isfinite().any() and torch.equal(got[[0, 1, 6, 7]], clean[[0, 1, 6, 7]])


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("inter", [300, 416])
def test_an_infinite_scale_of_a_row_s_last_block(inter, tokens):
    """The output that the block is part of is infinite, and no NaN comes from
    the k's behind the row's end."""
    layer = Layer(E4M3, 2, 64, inter, 1)
    x, ids, w = tokens_of(tokens, 1, 2, 64, 3)
    ids[:] = 1
    clean = layer(x, ids, w)
    layer.s["down"].view(2, 64, -1)[1, 10, -1] = float("inf")
    got = layer(x, ids, w)
    assert got[:, 10].isinf().all()
    got[:, 10] = clean[:, 10]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("fmt", FORMATS)
def test_wide_rows_of_few_tokens(fmt):
    """Sixteen rows of down a workgroup (hidden from 4096 on), the last partial."""
    hidden = 4128 if fmt == MX8 else 4101
    layer = Layer(fmt, 3, hidden, 64, 2)
    for dtype in (torch.bfloat16, torch.float32):
        check(layer, *tokens_of(2, 2, 3, hidden, 1), dtype)


def test_scales_at_the_ends_of_e8m0():
    """Scales of 2^-127 and 2^127 as the codec decodes them."""
    layer = Layer(MX8, 2, 64, 32, 1)
    x, ids, w = tokens_of(2, 1, 2, 64, 3)
    ids[:, 0] = torch.tensor([0, 1])
    layer.s["down"].view(2, 64, 1)[0, 10] = 0
    out = layer(x, ids, w, out_dtype=torch.float32)
    assert float(out[0, 10].abs()) < 448 * 2.0 ** -110
    layer.s["down"].view(2, 64, 1)[0, 10] = 254
    layer.t["down"][0, 10] = 0
    layer.t["down"][0, 10, 3] = 0x38        # 1.0 * 2^127
    big = layer(x, ids, w, out_dtype=torch.float32)
    assert torch.equal(big[1], out[1])
    h = ref.silu(layer.v["gate"][0] @ x[0].double().cpu().numpy()) * (layer.v["up"][0] @ x[0].double().cpu().numpy())
    want = h[3] * 2.0 ** 127 * float(w[0, 0])
    assert abs(float(big[0, 10]) - want) <= 1e-4 * abs(want)


def test_empty_calls_and_given_buffers():
    dev = require_gpu()
    layer = Layer(MX8, 4, 64, 32, 1)
    x, ids, w = tokens_of(5, 2, 4, 64, 3)
    want = layer(x, ids, w)
    out = torch.full((6, 64), 3.0, device=dev, dtype=torch.bfloat16)
    ws = torch.zeros(fq.fp8q_moe_experts_workspace(5, 2, 4, 64, 32) + 64, dtype=torch.uint8, device=dev)
    ws[-64:] = 99
    got = layer(x, ids, w, out=out[:5], workspace=ws[:-64])
    assert got.data_ptr() == out.data_ptr() and torch.equal(out[:5], want)
    assert (out[5] == 3).all() and (ws[-64:] == 99).all()
    assert layer(*tokens_of(0, 2, 4, 64, 3)).shape == (0, 64)
    nothing = Layer(BF16, 4, 64, 0, 1)
    assert not nothing(x, ids, w).any()
    assert Layer(BF16, 4, 0, 16, 1)(x[:, :0].contiguous(), ids, w).shape == (5, 0)
    assert fq.fp8q_moe_experts_workspace(5, 2, 4, 64, 32, torch.float32) == 3 * 2 * 10 * 32


@pytest.mark.parametrize("fmt", FORMATS)
def test_experts_past_two_to_the_31_elements(fmt):
    """The last of many experts, whose rows start far into the array."""
    dev = require_gpu()
    E, I, H = 1024, 768, 2816
    n = E * I * H
    assert n > 2 ** 31
    layer = Layer(fmt, 1, H, I, 4)
    big = Layer.__new__(Layer)
    big.fmt, big.t, big.s = fmt, dict(layer.t), dict(layer.s)
    x, ids, w = tokens_of(2, 1, 1, H, 3)
    want = layer(x, ids, w)
    for k in ("gate", "up", "down"):
        rows, width = (H, I) if k == "down" else (I, H)
        t = torch.zeros(E, rows, width, dtype=layer.t[k].dtype, device=dev)
        t[-1] = layer.t[k][0]
        big.t[k] = t
        if fmt != BF16:
            s = torch.zeros(E * rows, layer.s[k].shape[-1], dtype=layer.s[k].dtype, device=dev)
            s[-rows:] = layer.s[k]
            big.s[k] = s
    assert torch.equal(big(x, torch.full_like(ids, E - 1), w), want)


def test_refusals():
    dev = require_gpu()
    layer = Layer(MX8, 4, 64, 32, 1)
    x, ids, w = tokens_of(5, 2, 4, 64, 3)
    t, s = layer.t, layer.s

    def call(x=x, ids=ids, w=w, gate=t["gate"], up=t["up"], down=t["down"], gs=s["gate"], us=s["up"], ds=s["down"], **k):
        return fq.fp8q_moe_experts(x, ids, w, gate, up, down, gate_scales=gs, up_scales=us, down_scales=ds, **k)
    bf = t["gate"].to(torch.bfloat16)
    for bad in (dict(x=x[0]), dict(x=x[:4]), dict(w=w[:4]), dict(ids=ids[:, :0], w=w[:, :0]),
                dict(gate=t["gate"][:3]), dict(up=t["up"][:, :16]), dict(down=t["gate"]), dict(gs=s["gate"][:-1]),
                dict(gate=t["gate"].transpose(1, 2).contiguous().transpose(1, 2)), dict(gate=bf), dict(gate=bf, gs=None),
                dict(us=s["up"].view(4, 32, 2)[:, ::2].expand(4, 16, 2)), dict(x=x.T.contiguous().T),
                dict(ds=torch.zeros(4 * 64, 1, device=dev)), dict(out=x[:4]), dict(workspace=torch.zeros(8, dtype=torch.uint8, device=dev)),
                dict(x=x.cpu()), dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(x=x.float()), dict(ids=ids.float()), dict(w=w.bfloat16()), dict(gate=t["gate"].float()),
                dict(gs=None), dict(gs=s["gate"].int()), dict(out=x.float())):
        with pytest.raises(TypeError):
            call(**bad)
    many = torch.zeros(1025, 1, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError, match="1024"):
        call(x=torch.zeros(1025, 64, dtype=torch.bfloat16, device=dev), ids=many, w=many.float())
    with pytest.raises(ValueError, match="multiples of 32"):
        l = Layer(BF16, 4, 48, 32, 1)
        fq.fp8q_moe_experts(x[:, :48].contiguous(), ids, w, l.t["gate"].to(torch.uint8), l.t["up"].to(torch.uint8),
                            l.t["down"].to(torch.uint8), gate_scales=s["gate"], up_scales=s["up"], down_scales=s["down"])
    with pytest.raises(fq.Fp8qError):
        call(out=x)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tokens,topk", [(24, 1), (25, 1), (13, 5), (75, 8), (16, 64), (1024, 1)])
def test_experts_without_rows_give_zeros(fmt, tokens, topk):
    """inter == 0 with few pairs and many, up to the most that there may be."""
    layer = Layer(fmt, 70, 96, 0, 1)
    x, ids, w = tokens_of(tokens, topk, 70, 96, 2, gone=0.1)
    w[0] = float("nan")                     # times no y
    assert fq.fp8q_moe_experts_workspace(tokens, topk, 70, 96, 0) == 0
    for dtype in (torch.bfloat16, torch.float32):
        buffer = torch.full((tokens + 1, 96), 3.0, device=x.device, dtype=dtype)
        layer(x, ids, w, out_dtype=dtype, out=buffer[:tokens])
        assert not buffer[:tokens].view(torch.uint8).any() and (buffer[tokens] == 3).all()


def at_an_odd_address(t):
    """A copy that begins as far off 16 bytes as its type allows."""
    wide = torch.empty(t.numel() + 1, dtype=t.dtype, device=t.device)
    wide[1:] = t.reshape(-1)
    return wide[1:].view(t.shape)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("hidden,inter", [(256, 512), (160, 96), (32, 2144)])
@pytest.mark.parametrize("tokens", [2, 9, 40, 200])
def test_rows_at_any_address(fmt, hidden, inter, tokens):
    """The same bits from matrices that do not begin at a multiple of 16 bytes,
    all three of them or one."""
    layer = Layer(fmt, 3, hidden, inter, 5)
    x, ids, w = tokens_of(tokens, 2, 3, hidden, tokens, gone=0.1)
    for dtype in (torch.bfloat16, torch.float32):
        want = check(layer, x, ids, w, dtype)
        for moved in (("gate", "up", "down"), ("gate",), ("up",), ("down",)):
            other = Layer.__new__(Layer)
            other.fmt, other.s = fmt, dict(layer.s)
            other.t = {k: at_an_odd_address(t) if k in moved else t for k, t in layer.t.items()}
            assert all(other.t[k].data_ptr() % 16 for k in moved)
            if fmt == MX8:
                other.s = {k: at_an_odd_address(s) if k in moved else s for k, s in layer.s.items()}
            assert torch.equal(other(x, ids, w, out_dtype=dtype), want), moved


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("name", ["gate", "up", "down"])
def test_a_block_of_the_smallest_e8m0_scale(name, tokens):
    """Codes of 8 and more times 2^-127 are past 2^-126: their values count.
    Another matrix's 2^60 keeps what comes of them far from there."""
    layer = Layer(MX8, 2, 64, 32, 1)
    x, ids, w = tokens_of(tokens, 1, 2, 64, 3)
    x = torch.where(x < 0, x - 1, x + 1)
    rng = np.random.default_rng(4)
    other = "down" if name == "up" else "up"
    layer.s[other] += 60
    layer.v[other] = layer.v[other] * 2.0 ** 60
    rows, width = layer.t[name].shape[1:]
    codes = (rng.integers(0x50, 0x7F, size=(rows, width)) | rng.integers(0, 2, size=(rows, width)) << 7).astype(np.uint8)
    layer.t[name][0] = torch.from_numpy(codes).to(x.device)
    layer.s[name].view(2, rows, -1)[0] = 0
    layer.v[name][0] = oracle.fp8_decode(codes, 0).astype(np.float64) * 2.0 ** -127
    for dtype in (torch.bfloat16, torch.float32):
        got = check(layer, x, ids, w, dtype)
        assert bool((got[ids[:, 0] == 0] != 0).all())


@pytest.mark.parametrize("tokens", [2, 40])
def test_mx8_values_past_fp32_are_infinite(tokens):
    """As mx8_dequantize decodes them; the largest below keeps its value."""
    layer = Layer(MX8, 2, 64, 32, 1)
    x, ids, w = tokens_of(tokens, 1, 2, 64, 3)
    ids[:] = 0
    clean = layer(x, ids, w, out_dtype=torch.float32)
    layer.t["down"][0, 10:12] = 0
    layer.t["down"][0, 10, 3] = 0x7E        # 448 * 2^120 = 1.75 * 2^128
    layer.t["down"][0, 11, 3] = 0x77        # 240 * 2^120
    layer.s["down"].view(2, 64, 1)[0, 10:12] = 247
    w = w * 2.0 ** -10
    got = layer(x, ids, w, out_dtype=torch.float32)
    values = fq.mx8_dequantize(layer.t["down"].view(128, 32), layer.s["down"].view(128, 1)).view(2, 64, 32)
    h = ref.silu(layer.v["gate"][0] @ x.double().cpu().numpy().T) * (layer.v["up"][0] @ x.double().cpu().numpy().T)
    assert values[0, 10, 3].isinf() and float(values[0, 11, 3]) == 240.0 * 2.0 ** 120
    for i, h3 in enumerate(h[3]):
        assert not np.isfinite(float(got[i, 10]))
        want = 240.0 * 2.0 ** 120 * h3 * float(w[i, 0])
        if abs(want) < 2.0 ** 117:
            assert abs(float(got[i, 11]) - want) <= 1e-4 * abs(want)
    keep = [c for c in range(64) if c not in (10, 11)]
    assert torch.equal(got[:, keep], clean[:, keep] * 2.0 ** -10)


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("width", [64, 200])
@pytest.mark.parametrize("fmt", FORMATS[1:3])
def test_scales_far_from_one(fmt, width, tokens):
    """A power of two taken from x and put into the scales, or from one matrix's
    scales and put into the next one's, changes no bit: neither code * x nor code
    * h has to be in fp32's range where code * scale * x is."""
    experts, dev = 2, require_gpu()
    x, ids, w = tokens_of(tokens, 1, experts, width, 3)
    x = torch.where(x < 0, x - 1, x + 1)
    g = torch.Generator().manual_seed(7)

    def layer(codes, size):
        made = Layer.__new__(Layer)
        made.fmt, made.t, made.s = fmt, {}, {}
        for k in ("gate", "up", "down"):
            q = codes[torch.randint(0, len(codes), (experts, width, width), generator=g)]
            q = q | (torch.randint(0, 2, q.shape, generator=g) << 7)
            made.t[k] = q.to(torch.uint8).to(dev)
            made.s[k] = (size * (1 + torch.rand(experts * width, -(-width // 128), generator=g))).to(dev)
        return made

    def times(layer, **powers):
        made = Layer.__new__(Layer)
        made.fmt, made.t, made.s = fmt, layer.t, dict(layer.s)
        for k, p in powers.items():
            made.s[k] = layer.s[k] * 2.0 ** p
        return made

    # the largest codes: 448, or 57344 (x times 2^k, h times 2^100 and more)
    for codes, size, k, p in ((torch.tensor([0x7E, 0x7D] if fmt == E4M3 else [0x7B, 0x7A]), 2.0 ** -5, 120, 100),
                              # the smallest: 2^-9, or 2^-16
                              (torch.tensor([1, 2, 3]), 2.0 ** (6 if fmt == E4M3 else 13), -120, -90)):
        if fmt == E5M2:
            size, k, p = (2.0 ** -12, 113, 95) if k > 0 else (size, -110, p)
        made = layer(codes, size)
        for dtype in (torch.bfloat16, torch.float32):
            want = made(x, ids, w, out_dtype=dtype)
            assert want.isfinite().all() and (want != 0).any()
            moved = times(made, gate=-k, up=-k)
            assert torch.equal(moved(x * 2.0 ** k, ids, w, out_dtype=dtype), want)
            moved = times(made, up=p, down=-p)
            assert torch.equal(moved(x, ids, w, out_dtype=dtype), want)


@pytest.mark.parametrize("tokens", [2, 40])
@pytest.mark.parametrize("fmt", FORMATS[1:3])
def test_subnormal_scales(fmt, tokens):
    layer = Layer(fmt, 2, 96, 200, 1)
    x, ids, w = tokens_of(tokens, 1, 2, 96, 3)
    layer.s["down"].fill_(2.0 ** -30)
    want = layer(x, ids, w, out_dtype=torch.float32)
    layer.s["up"] *= 2.0 ** 110
    layer.s["down"].fill_(2.0 ** -140)
    got = layer(x, ids, w, out_dtype=torch.float32)
    assert bool((want != 0).any()) and torch.equal(got, want)
