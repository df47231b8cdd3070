"""The norm of gradients and their clipping on the GPU: sums against exactly
rounded ones, clipped values bit for bit."""
import math

import numpy as np
import pytest
import torch

import dequantize_reduce_transfer_amd as fq
import model_ref as ref
import oracle
from gpu_util import host, require_gpu

pytestmark = pytest.mark.gpu

# A sum of squares: every term is exact in fp64 and none is negative, so n
# additions in any order are off by at most n * 2^-53 of the sum.
def sum_bound(n):
    return (n + 2) * 2.0 ** -53


# sizes around a vector, a block of codes, a chunk and several workgroups
SIZES = [1, 3, 15, 16, 17, 127, 128, 129, 1000, 1023, 1024, 1025, 4096, 4097, 70001]


def gradient(kind, n, seed, offset=0):
    """(tensor, scales, fp32 values); the tensor a view at an odd offset."""
    rng = np.random.default_rng(seed)
    dev = require_gpu()
    if kind in ("f32", "bf16"):
        t = torch.from_numpy(rng.normal(size=n + offset).astype(np.float32)).to(dev)
        t = (t if kind == "f32" else t.bfloat16())[offset:]
        return t, None, t.float().cpu().numpy()
    fmt = {"e4m3": 0, "e5m2": 1, "tensorwise": 0, "tensorwise5": 1}[kind]
    codes = rng.integers(0, 256, size=n + offset, dtype=np.uint8)
    codes[np.isnan(oracle.fp8_decode(codes, fmt)) | np.isinf(oracle.fp8_decode(codes, fmt))] = 0
    blocks = 1 if kind.startswith("tensorwise") else -(-n // 128)
    scales = np.exp(rng.normal(size=blocks + offset)).astype(np.float32)
    v = oracle.fp8_decode(codes[offset:], fmt).astype(np.float32)
    s = scales[offset:]
    v = (v * (s if blocks == 1 else s.repeat(128)[:n])).astype(np.float32)
    return torch.from_numpy(codes).to(dev)[offset:], torch.from_numpy(scales).to(dev)[offset:], v


def fmt_of(kind):
    return fq.E5M2 if kind in ("e5m2", "tensorwise5") else fq.E4M3


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "e5m2", "tensorwise", "tensorwise5"])
def test_sum_of_each_size(kind):
    for i, n in enumerate(SIZES):
        for offset in (0, 1, 3):
            t, s, v = gradient(kind, n, i, offset)
            got = fq.fp8q_grad_sumsq([t], scales=[s], fmt=fmt_of(kind))
            assert got.dtype == torch.float64 and got.shape == (1,)
            want = ref.sumsq([v])
            assert abs(float(got) - want) <= sum_bound(n) * want, (n, offset)


def coefficient(sumsq, max_norm, eps=1e-6):
    with np.errstate(all="ignore"):
        return np.float32(min(1.0, np.float64(max_norm) / (np.sqrt(np.float64(sumsq)) + np.float64(eps))))


def clipped(t, s, by):
    """What clipping leaves, from what was there (by torch on the CPU: products
    of fp32, rounded once)."""
    if s is not None:
        return s.cpu() * torch.tensor(by)
    return (t.cpu().float() * torch.tensor(by)).to(t.dtype)


@pytest.mark.parametrize("kind", ["f32", "bf16", "e4m3", "tensorwise5"])
def test_clip_of_each_size(kind):
    for i, n in enumerate(SIZES):
        for offset in (0, 1, 3):
            t, s, v = gradient(kind, n, i, offset)
            dev, total = t.device, torch.tensor([7.3], dtype=torch.float64)
            codes = t.clone()
            want = clipped(t, s, coefficient(7.3, 1.0))
            norm = fq.fp8q_grad_clip([t], total.to(dev), 1.0, scales=[s], fmt=fmt_of(kind))
            assert float(norm) == float(np.float32(math.sqrt(7.3))) and norm.shape == (1,)
            assert torch.equal((t if s is None else s).cpu(), want), (n, offset)
            if s is not None:
                assert torch.equal(t, codes)


def views(kinds, count, seed):
    """A list of views of one buffer a kind, side by side, and sentinels behind
    each buffer's last one."""
    rng = np.random.default_rng(seed)
    out = []
    for i in range(count):
        kind = kinds[i % len(kinds)]
        out.append((kind, int(rng.integers(1, 300) if i % 7 else rng.integers(3000, 20000))))
    flat = {k: sum(n for q, n in out if q == k) for k in kinds}
    dev = require_gpu()
    whole, at = {}, {k: 0 for k in kinds}
    for k in kinds:
        w = torch.from_numpy(rng.normal(size=flat[k] + 5).astype(np.float32)).to(dev)
        whole[k] = w if k == "f32" else w.bfloat16()
    grads = []
    for k, n in out:
        grads.append(whole[k][at[k]:at[k] + n])
        at[k] += n
    return grads, whole, flat


@pytest.mark.parametrize("count", [1, 2, 31, 32, 33, 159, 160, 161, 249, 250, 251, 520])
def test_many_tensors(count):
    kinds = ["f32", "bf16"] if count > 1 else ["bf16"]
    grads, whole, flat = views(kinds, count, count)
    before = {k: w.clone() for k, w in whole.items()}
    want = ref.sumsq([g.float().cpu().numpy() for g in grads])
    total = fq.fp8q_grad_sumsq(tuple(grads))
    assert abs(float(total) - want) <= sum_bound(sum(flat.values())) * want
    assert all(torch.equal(fq.fp8q_grad_sumsq(grads), total) for _ in range(3))
    assert all(torch.equal(whole[k], before[k]) for k in kinds)
    by = coefficient(float(total), 0.37)
    norm = fq.fp8q_grad_clip(grads, total, 0.37)
    assert float(norm) == float(np.float32(math.sqrt(float(total))))
    for k in kinds:
        assert torch.equal(whole[k][:flat[k]].cpu(), clipped(before[k][:flat[k]], None, by))
        assert torch.equal(whole[k][flat[k]:], before[k][flat[k]:])


def test_a_mixed_list_with_codes_and_empty_ones():
    dev = require_gpu()
    made = [gradient(k, n, i, i % 3) for i, (k, n) in enumerate(
        [("f32", 1000), ("e4m3", 777), ("bf16", 513), ("tensorwise", 300), ("f32", 1), ("e4m3", 128), ("bf16", 65537)])]
    empty = [(torch.zeros(0, device=dev), None), (torch.zeros(0, dtype=torch.uint8, device=dev), torch.zeros(0, device=dev))]
    grads = [t for t, _, _ in made] + [t for t, _ in empty]
    scales = [s for _, s, _ in made] + [s for _, s in empty]
    total = fq.fp8q_grad_sumsq(grads, scales=scales)
    want = ref.sumsq([v for _, _, v in made])
    assert abs(float(total) - want) <= sum_bound(70000) * want
    by = coefficient(float(total), 2.0)
    wants = [clipped(t, s, by) for t, s, _ in made]
    fq.fp8q_grad_clip(grads, total, 2.0, scales=scales)
    for (t, s, _), w in zip(made, wants):
        assert torch.equal((t if s is None else s).cpu(), w)
    # and once more: the norm is at the limit now
    again = fq.fp8q_grad_sumsq(grads, scales=scales)
    assert abs(math.sqrt(float(again)) - 2.0) < 2.0 * 2 ** -8


def test_nothing_is_written_within_the_limit():
    dev = require_gpu()
    t = torch.tensor([3.0, 4.0, math.nan, -0.0], device=dev)
    for total, limit in ((25.0, 5.1), (0.0, 0.0001), (25.0, math.inf), (math.nan, math.inf), (math.inf, math.inf)):
        keep = t.clone()
        norm = fq.fp8q_grad_clip([t], torch.tensor([total], dtype=torch.float64, device=dev), limit)
        assert torch.equal(t.view(torch.int32), keep.view(torch.int32))
        np.testing.assert_equal(float(norm), math.sqrt(total) if total == total else math.nan)


def test_special_norms():
    dev = require_gpu()
    start = torch.tensor([3.0, -4.0, math.inf, math.nan, 0.0], device=dev)
    for dtype in (torch.float32, torch.bfloat16):
        for total, want in ((math.nan, [math.nan] * 5), (math.inf, [0.0, -0.0, math.nan, math.nan, 0.0])):
            t = start.to(dtype, copy=True)
            fq.fp8q_grad_clip([t], torch.tensor([total], dtype=torch.float64, device=dev), 1.0)
            np.testing.assert_equal(t.float().cpu().numpy(), np.array(want, np.float32))
    t = start[:2].clone()
    fq.fp8q_grad_clip([t], torch.tensor([25.0], dtype=torch.float64, device=dev), 0.0)
    assert t.tolist() == [0.0, -0.0]
    t = start[:2].clone()                # eps 0, norm 0: 0 / 0
    fq.fp8q_grad_clip([t], torch.zeros(1, dtype=torch.float64, device=dev), 0.0, eps=0.0)
    assert t.isnan().all()
    for bad in (math.nan, math.inf, -math.inf):
        g = torch.ones(5000, device=dev)
        g[4321] = bad
        np.testing.assert_equal(float(fq.fp8q_grad_sumsq([g])), math.nan if bad != bad else math.inf)


def test_the_range_of_fp32():
    """Squares that fp32 does not hold."""
    dev = require_gpu()
    for v in (3e38, 1e-30, 1e-45):
        t = torch.full((3000,), v, device=dev)
        x = float(t[0])
        assert abs(float(fq.fp8q_grad_sumsq([t])) - 3000 * x * x) <= sum_bound(3000) * 3000 * x * x
    t = torch.full((300,), 3e38, device=dev)
    norm = fq.fp8q_grad_clip([t], fq.fp8q_grad_sumsq([t]), 1.0)
    assert float(norm) == math.inf       # past fp32 itself; the values are scaled all the same
    assert abs(float(t[0]) - 1 / math.sqrt(300)) < 1e-6


@pytest.mark.parametrize("n", [1 << 20, (1 << 23) + 11, (1 << 27) + 5])
def test_large_tensors(n):
    """Each chunk size; the sum of equal values is exact arithmetic."""
    dev = require_gpu()
    for dtype in (torch.float32, torch.bfloat16):
        t = torch.full((n,), 0.5, device=dev, dtype=dtype)
        t[n // 3] = 96.0
        assert float(fq.fp8q_grad_sumsq([t])) == (n - 1) * 0.25 + 96.0 ** 2
        fq.fp8q_grad_clip([t], torch.tensor([16.0], dtype=torch.float64, device=dev), 1.0, eps=0.0)
        t[n // 3] *= 0.5 / 96.0
        assert bool((t == 0.125).all())
        del t


def test_past_two_to_the_32_bytes_and_elements():
    dev = require_gpu()
    n = (1 << 32) + 1027
    q = torch.zeros(n, dtype=torch.uint8, device=dev)
    q[-1] = q[1 << 32] = q[0] = 0x38     # 1.0
    s = torch.ones(-(-n // 128), device=dev)
    s[-1] = 3.0
    assert float(fq.fp8q_grad_sumsq([q], scales=[s])) == 1.0 + 1.0 + 9.0
    del q, s
    t = torch.zeros((1 << 31) + 77, dtype=torch.bfloat16, device=dev)
    t[-1] = 2.0
    assert float(fq.fp8q_grad_sumsq([t])) == 4.0
    fq.fp8q_grad_clip([t], torch.tensor([4.0], dtype=torch.float64, device=dev), 1.0, eps=0.0)
    assert float(t[-1]) == 1.0 and not t[:-1].any()


def test_empty_lists_and_given_outputs():
    dev = require_gpu()
    out = torch.full((1,), 5.0, dtype=torch.float64, device=dev)
    assert fq.fp8q_grad_sumsq([], out=out).data_ptr() == out.data_ptr() and float(out) == 0.0
    assert float(fq.fp8q_grad_sumsq([torch.zeros(0, device=dev)])) == 0.0
    norm = torch.zeros(2, device=dev)
    fq.fp8q_grad_clip([], torch.tensor([9.0], dtype=torch.float64, device=dev), 1.0, norm_out=norm[:1])
    assert norm.tolist() == [3.0, 0.0]
    g = [torch.ones(100000, device=dev) for _ in range(3)]
    ws = torch.zeros(16384, dtype=torch.uint8, device=dev)
    assert float(fq.fp8q_grad_sumsq(g, workspace=ws)) == 300000.0
    with pytest.raises(ValueError, match="workspace"):
        fq.fp8q_grad_sumsq(g, workspace=ws[:16])


def test_refusals():
    dev = require_gpu()
    t, total = torch.ones(64, device=dev), torch.ones(1, dtype=torch.float64, device=dev)
    q, s = torch.zeros(300, dtype=torch.uint8, device=dev), torch.ones(3, device=dev)
    for bad in (lambda: fq.fp8q_grad_sumsq([t.view(8, 8).T]), lambda: fq.fp8q_grad_sumsq([t], scales=[s]),
                lambda: fq.fp8q_grad_sumsq([q], scales=[s[:2]]), lambda: fq.fp8q_grad_sumsq([t], scales=[None, None]),
                lambda: fq.fp8q_grad_clip([t], total.view(1, 1), 1.0), lambda: fq.fp8q_grad_sumsq([t], out=total.expand(2)),
                lambda: fq.fp8q_grad_sumsq([t, t.cpu()]), lambda: fq.fp8q_grad_clip([t], total, 1.0, norm_out=t)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fq.fp8q_grad_sumsq([q]), lambda: fq.fp8q_grad_sumsq([t.half()]), lambda: fq.fp8q_grad_sumsq(t),
                lambda: fq.fp8q_grad_clip([t], total.float(), 1.0), lambda: fq.fp8q_grad_clip([t], total, "x"),
                lambda: fq.fp8q_grad_sumsq([q], scales=[q])):
        with pytest.raises(TypeError):
            bad()
    keep = t.clone()
    for bad in (lambda: fq.fp8q_grad_clip([t, t], total, 0.5), lambda: fq.fp8q_grad_clip([t, t[5:9]], total, 0.5),
                lambda: fq.fp8q_grad_clip([t], total, -1.0), lambda: fq.fp8q_grad_clip([t], total, math.nan),
                lambda: fq.fp8q_grad_clip([t], total, 1.0, eps=-1.0),
                lambda: fq.fp8q_grad_clip([q, q], total, 1.0, scales=[s, s]),
                lambda: fq.fp8q_grad_clip([t], total, 1.0, norm_out=t[3:4])):
        with pytest.raises(fq.Fp8qError):
            bad()
    assert torch.equal(t, keep)
    assert float(fq.fp8q_grad_sumsq([t, t])) == 128.0    # reading twice is no harm


def test_clipping_is_an_in_place_change_to_autograd():
    dev = require_gpu()
    total = torch.tensor([100.0], dtype=torch.float64, device=dev)
    x = torch.arange(1.0, 5.0, device=dev, requires_grad=True)
    g, = torch.autograd.grad((x ** 3).sum(), x, create_graph=True)
    penalty = (g * g).sum()                 # saves g
    fq.fp8q_grad_clip([g.detach()], total, 1.0)
    with pytest.raises(RuntimeError, match="inplace"):
        penalty.backward()
    q, s = torch.zeros(300, dtype=torch.uint8, device=dev), torch.ones(3, device=dev)
    t, b = torch.ones(7, device=dev), torch.ones(9, dtype=torch.bfloat16, device=dev)
    before = [v._version for v in (t, q, s, b)]
    fq.fp8q_grad_clip([t, q, b], total, 1.0, scales=[None, s, None])
    assert [v._version - n for v, n in zip((t, q, s, b), before)] == [1, 0, 1, 1]
    fq.fp8q_grad_clip((t,), total, 1.0, stream=torch.cuda.Stream(dev))
    torch.cuda.synchronize()
    assert t._version == before[0] + 2
    fq.fp8q_grad_sumsq([t, q, b], scales=[None, s, None])
    with pytest.raises(fq.Fp8qError):
        fq.fp8q_grad_clip([t], total, -1.0)
    assert t._version == before[0] + 2
    with torch.inference_mode():
        i = torch.ones(5, device=dev)
        fq.fp8q_grad_clip([i], total, 1.0, eps=0.0)
    fq.fp8q_grad_clip([i], total, 1.0, eps=0.0)
    assert bool((i == torch.full((5,), 0.1, device=dev) * torch.tensor(0.1)).all())


def test_a_number_that_changes_the_list():
    """What the lists hold when the tensors are taken is what is clipped."""
    dev = require_gpu()
    total = torch.tensor([100.0], dtype=torch.float64, device=dev)
    kept = torch.ones(1000, device=dev)
    grads = [kept, torch.ones(5000, device=dev)]

    class Clears:
        def __float__(self):
            grads.clear()
            return 1.0

    assert float(fq.fp8q_grad_clip(grads, total, Clears())) == 10.0
    grads.append(torch.ones(5000, device=dev))
    assert float(fq.fp8q_grad_clip(grads, total, 1.0, eps=Clears())) == 10.0
    assert not grads and bool((kept == 1).all())
