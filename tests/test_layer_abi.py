"""The C ABI of include/fp8q_layer.h: the library exports what the header
declares, and rejects every bad request on the host before any launch; the
Python functions refuse tensors that do not fit.

The validation tests never reach a launch: each call fails first.  They are
skipped when a GPU is visible, so that a validation bug could never turn a host
pointer into a launch there.  tests/test_layer_abi_sanitized.py runs this file
against a host-check build whose launchers are stubs, where accepted calls can
run too.
"""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import dequantize_reduce_transfer_amd as fq
from dequantize_reduce_transfer_amd import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8q_layer.h")
LIB = os.environ.get("FP8Q_LAYER_HOSTCHECK", layer.LIB_PATH)

OK, ERR_NULL, ERR_ARG, ERR_ALIGN, ERR_OVERLAP, ERR_HIP = range(6)

no_gpu = pytest.mark.skipif(torch.cuda.device_count() > 0,
                            reason="host-only validation tests; a GPU is visible")


def L():
    return layer.layer_lib(LIB)


class Buf:
    """Host memory whose addresses stand in for device pointers."""

    def __init__(self, nbytes):
        self.raw = ctypes.create_string_buffer(int(nbytes) + 64)
        self.addr = (ctypes.addressof(self.raw) + 15) // 16 * 16


def P(x):
    return ctypes.c_void_p(x)


def _declared():
    return sorted(re.findall(r"^FP8Q_API\s+\w+\s+(\w+)\s*\(", open(HEADER).read(), re.M))


def test_header_declares_the_abi():
    assert _declared() == sorted(layer.EXPORTS)
    text = open(HEADER).read()
    assert re.search(r"#define FP8Q_NORM_MAX_HIDDEN %d\b" % layer.NORM_MAX_HIDDEN, text)
    assert re.search(r"#define FP8Q_MAX_TOPK %d\b" % layer.MAX_TOPK, text)
    assert re.search(r"#define FP8Q_MAX_EXPERTS %d\b" % layer.MAX_EXPERTS, text)
    assert layer.MAX_HIDDEN == 1 << 20 and "FP8Q_MAX_HIDDEN (((size_t)1) << 20)" in text


def test_library_exports_exactly_what_is_declared():
    out = subprocess.run(["nm", "-D", "--defined-only", layer.LIB_PATH], capture_output=True, text=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if " T " in line} == set(_declared())


def test_header_compiles_as_c():
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), "-x", "c", "-"],
                       input='#include "fp8q_layer.h"\nint main(void) { return FP8Q_MAX_TOPK == 64 ? 0 : 1; }\n',
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_library_holds_no_kernel_that_no_size_reaches():
    """Rows of under eight elements (Edge 2) have one shape: a wave, a vector."""
    names = re.findall(rb"\d+(norm\w*?_kernel)I\w*?LNS_4EdgeE2ELi(\d+)ELi(\d+)E", open(layer.LIB_PATH, "rb").read())
    assert {(kernel.decode(), int(w), int(v)) for kernel, w, v in names} == {
        (kernel, 1, 1) for kernel in ("norm_kernel", "norm_backward_kernel", "norm_backward_columns_kernel")}


NORM = dict(x=0, res=1, w=2, wt=3, eps=4, rows=5, hidden=6, fmt=7, h=8, y=9, q=10, s=11, rstd=12)


def norm_args(mx=False, rows=4, hidden=256):
    n = rows * hidden
    bufs = dict(x=Buf(2 * n), res=Buf(2 * n), w=Buf(4 * hidden), h=Buf(2 * n), y=Buf(2 * n), q=Buf(n),
                s=Buf(n), rstd=Buf(4 * rows))
    args = dict(x=P(bufs["x"].addr), res=P(bufs["res"].addr), w=P(bufs["w"].addr), wt=1, eps=1e-6,
                rows=rows, hidden=hidden, fmt=0, h=P(bufs["h"].addr), y=P(bufs["y"].addr),
                q=P(bufs["q"].addr), s=P(bufs["s"].addr), rstd=P(bufs["rstd"].addr))

    def call(**change):
        a = dict(args, **change)
        order = [k for k in NORM if not (mx and k == "fmt")]
        return (L().mx8_rms_norm_quantize if mx else L().fp8q_rms_norm_quantize)(*[a[k] for k in order], None)
    call.bufs, call.addr = bufs, lambda k, off=0: P(bufs[k].addr + off)
    return call


@no_gpu
@pytest.mark.parametrize("mx", [False, True])
def test_norm_validation(mx):
    c = norm_args(mx)
    for bad in (dict(wt=2), dict(wt=-1), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")),
                dict(hidden=32768 + 32), dict(rows=1 << 40), dict(res=None),
                *([dict(hidden=48)] if mx else [dict(fmt=2), dict(fmt=-1)])):
        assert c(**bad) == ERR_ARG, bad
    assert c(rows=0) == OK and c(hidden=0) == OK and c(x=None, rows=0) == OK
    for k in ("x", "w", "q", "s"):
        assert c(**{k: None}) == ERR_NULL, k
    for k in ("x", "res", "w", "h", "y", "q"):
        assert c(**{k: c.addr(k, 8)}) == ERR_ALIGN, k
    assert c(rstd=c.addr("rstd", 2)) == ERR_ALIGN
    if not mx:
        assert c(s=c.addr("s", 2)) == ERR_ALIGN
    n = 4 * 256
    for k, at in [("q", c.addr("x", 2 * n - 16)), ("q", c.addr("res")), ("y", c.addr("h", 16)),
                  ("y", c.addr("x")), ("h", c.addr("x", 16)), ("h", c.addr("res", 2 * n - 16)),
                  ("s", c.addr("q", n - 4)), ("rstd", c.addr("s")), ("rstd", c.addr("w", 16)),
                  ("h", c.addr("q")), ("y", c.addr("w"))]:
        assert c(**{k: at}) == ERR_OVERLAP, (k, at)
    # the residual updated in place, but another input in the way
    assert c(h=c.addr("res"), x=c.addr("res", 16)) == ERR_OVERLAP


BACK = ["dy", "h", "w", "wt", "rstd", "dh", "rows", "hidden", "dx", "dw", "ws", "wsb"]


def back_args(rows=40, hidden=64):
    n = rows * hidden
    need = L().fp8q_rms_norm_backward_workspace(rows, hidden)
    bufs = dict(dy=Buf(2 * n), h=Buf(2 * n), w=Buf(4 * hidden), rstd=Buf(4 * rows), dh=Buf(2 * n),
                dx=Buf(2 * n), dw=Buf(4 * hidden), ws=Buf(need))
    args = {k: P(b.addr) for k, b in bufs.items()}
    args.update(wt=0, rows=rows, hidden=hidden, wsb=need)

    def call(**change):
        a = dict(args, **change)
        return L().fp8q_rms_norm_backward(*[a[k] for k in BACK], None)
    call.addr, call.need = lambda k, off=0: P(bufs[k].addr + off), need
    return call


@no_gpu
def test_norm_backward_validation():
    c = back_args()
    assert c.need > 0
    for bad in (dict(wt=3), dict(hidden=40000), dict(rows=1 << 40), dict(wsb=c.need - 1)):
        assert c(**bad) == ERR_ARG, bad
    assert c(hidden=0) == OK
    for k in ("dy", "h", "w", "rstd", "dx", "dw", "ws"):
        assert c(**{k: None}) == ERR_NULL, k
    for k in ("dy", "h", "w", "dh", "dx", "ws"):
        assert c(**{k: c.addr(k, 4)}) == ERR_ALIGN, k
    assert c(rstd=c.addr("rstd", 1)) == ERR_ALIGN and c(dw=c.addr("dw", 2)) == ERR_ALIGN
    for k, at in [("dx", c.addr("h")), ("dx", c.addr("dy", 16)), ("dx", c.addr("dh", 32)), ("dw", c.addr("dy")),
                  ("dw", c.addr("dx", 64)), ("ws", c.addr("h")), ("dx", c.addr("ws"))]:
        assert c(**{k: at}) == ERR_OVERLAP, (k, at)
    assert L().fp8q_rms_norm_backward_workspace(0, 64) == 0
    assert L().fp8q_rms_norm_backward_workspace(40, 40000) == 0


@no_gpu
def test_sort_validation():
    tokens, topk, experts = 700, 8, 16
    n = tokens * topk
    need = L().fp8q_moe_sort_workspace(tokens, topk, experts)
    ids, slots, pairs, offs, ws = Buf(8 * n), Buf(4 * n), Buf(4 * n), Buf(4 * 17), Buf(need)
    base = dict(ids=P(ids.addr), w=4, t=tokens, k=topk, e=experts, s=P(slots.addr), p=P(pairs.addr),
                o=P(offs.addr), ws=P(ws.addr), wsb=need)

    def c(**change):
        a = dict(base, **change)
        return L().fp8q_moe_sort(*[a[k] for k in base], None)

    assert need > 0
    for bad in (dict(w=2), dict(w=0), dict(k=0), dict(k=65), dict(e=0), dict(e=1025), dict(t=1 << 30),
                dict(wsb=need - 1), dict(t=1 << 62)):
        assert c(**bad) == ERR_ARG, bad
    for k in ("ids", "s", "p", "o", "ws"):
        assert c(**{k: None}) == ERR_NULL, k
    assert c(ids=P(ids.addr + 4), w=8) == ERR_ALIGN and c(ids=P(ids.addr + 2)) == ERR_ALIGN
    assert c(s=P(slots.addr + 1)) == ERR_ALIGN and c(ws=P(ws.addr + 4)) == ERR_ALIGN
    for bad in (dict(s=P(ids.addr)), dict(p=P(slots.addr + 4 * n - 4)), dict(o=P(pairs.addr)),
                dict(ws=P(ids.addr)), dict(s=P(ws.addr))):
        assert c(**bad) == ERR_OVERLAP, bad
    assert L().fp8q_moe_sort_workspace(tokens, 0, experts) == 0
    assert L().fp8q_moe_sort_workspace(1 << 62, 8, experts) == 0


@no_gpu
def test_permute_validation():
    t, k, rb, sb, rows = 10, 4, 96, 12, 40
    src, ss, sl, dst, ds = Buf(t * rb), Buf(t * sb), Buf(4 * t * k), Buf(rows * rb), Buf(rows * sb)
    base = dict(src=P(src.addr), rb=rb, ss=P(ss.addr), sb=sb, sl=P(sl.addr), t=t, k=k, rows=rows,
                dst=P(dst.addr), ds=P(ds.addr))

    def c(**change):
        a = dict(base, **change)
        return L().fp8q_moe_permute(*[a[x] for x in base], None)

    for bad in (dict(k=0), dict(k=65), dict(t=1 << 62), dict(rows=(1 << 30) + 1), dict(rb=0),
                dict(rb=(1 << 22) + 1), dict(sb=(1 << 22) + 1)):
        assert c(**bad) == ERR_ARG, bad
    assert c(t=0) == OK and c(rows=0) == OK and c(rb=0, sb=0) == OK
    for x in ("src", "sl", "dst", "ss", "ds"):
        assert c(**{x: None}) == ERR_NULL, x
    assert c(src=P(src.addr + 8)) == ERR_ALIGN and c(dst=P(dst.addr + 4)) == ERR_ALIGN
    assert c(sl=P(sl.addr + 2)) == ERR_ALIGN
    for bad in (dict(dst=P(src.addr)), dict(ds=P(dst.addr + rows * rb - 1)), dict(ds=P(ss.addr)),
                dict(dst=P(sl.addr))):
        assert c(**bad) == ERR_OVERLAP, bad


@no_gpu
def test_combine_validation():
    t, k, hid, n = 6, 3, 128, 18
    rows, sc, sl, w, out = Buf(2 * n * hid), Buf(4 * n * 4), Buf(4 * t * k), Buf(4 * t * k), Buf(4 * t * hid)
    base = dict(rows=P(rows.addr), f=1, sc=P(sc.addr), sl=P(sl.addr), w=P(w.addr), t=t, k=k, n=n, hid=hid,
                out=P(out.addr), od=0)

    def c(**change):
        a = dict(base, **change)
        return L().fp8q_moe_combine(*[a[x] for x in base], None)

    for bad in (dict(f=4), dict(f=-1), dict(od=2), dict(k=0), dict(k=65), dict(t=1 << 62), dict(f=3, hid=40),
                dict(n=(1 << 30) + 1), dict(hid=(1 << 20) + 32)):
        assert c(**bad) == ERR_ARG, bad
    assert c(t=0) == OK and c(hid=0) == OK
    for x in ("rows", "sl", "sc", "out"):
        assert c(**{x: None}) == ERR_NULL, x
    assert c(rows=P(rows.addr + 8)) == ERR_ALIGN and c(out=P(out.addr + 8)) == ERR_ALIGN
    assert c(sc=P(sc.addr + 2)) == ERR_ALIGN and c(w=P(w.addr + 2)) == ERR_ALIGN
    for bad in (dict(out=P(rows.addr)), dict(out=P(sc.addr)), dict(w=P(out.addr + 16)), dict(sl=P(out.addr))):
        assert c(**bad) == ERR_OVERLAP, bad


@no_gpu
def test_combine_backward_validation():
    t, k, hid, n = 6, 3, 64, 18
    dy, rows, sl, w = Buf(2 * t * hid), Buf(2 * n * hid), Buf(4 * t * k), Buf(4 * t * k)
    dr, dw = Buf(2 * n * hid), Buf(4 * t * k)
    base = dict(dy=P(dy.addr), rows=P(rows.addr), sl=P(sl.addr), w=P(w.addr), t=t, k=k, n=n, hid=hid,
                dr=P(dr.addr), dw=P(dw.addr))

    def c(**change):
        a = dict(base, **change)
        return L().fp8q_moe_combine_backward(*[a[x] for x in base], None)

    for bad in (dict(k=0), dict(k=65), dict(t=1 << 62), dict(n=(1 << 30) + 1), dict(hid=(1 << 20) + 1)):
        assert c(**bad) == ERR_ARG, bad
    assert c(t=0) == OK
    for x in ("dy", "rows", "sl", "w", "dr", "dw"):
        assert c(**{x: None}) == ERR_NULL, x
    assert c(dy=P(dy.addr + 2)) == ERR_ALIGN and c(dr=P(dr.addr + 8)) == ERR_ALIGN
    assert c(dw=P(dw.addr + 1)) == ERR_ALIGN
    for bad in (dict(dr=P(rows.addr)), dict(dr=P(dy.addr)), dict(dw=P(w.addr)), dict(dw=P(dr.addr + 16))):
        assert c(**bad) == ERR_OVERLAP, bad


# Accepted calls, against the host-check build.

def _stub():
    if "FP8Q_LAYER_HOSTCHECK" not in os.environ:
        pytest.skip("needs the host-check build of the library (FP8Q_LAYER_HOSTCHECK)")
    S = L()
    S.layer_stub_calls.restype = ctypes.c_long
    S.layer_stub_last.restype = ctypes.c_char_p
    S.layer_stub_a.restype = S.layer_stub_b.restype = ctypes.c_ulonglong
    return S


def _launches(S, call, name, a, b):
    before = S.layer_stub_calls()
    assert call() == OK
    assert S.layer_stub_calls() == before + 1
    assert (S.layer_stub_last().decode(), S.layer_stub_a(), S.layer_stub_b()) == (name, a, b)


def test_accepted_calls_reach_their_launcher_once():
    S = _stub()
    for mx, name in ((False, "fp8q_rms_norm"), (True, "mx8_rms_norm")):
        c = norm_args(mx)
        _launches(S, c, name, 4, 256)
        _launches(S, lambda: c(res=None, h=None, y=None, rstd=None, eps=0.0), name, 4, 256)
        _launches(S, lambda: c(h=c.addr("res")), name, 4, 256)      # in place
        _launches(S, lambda: c(h=c.addr("x")), name, 4, 256)
    c = norm_args(False, 3, 33)
    _launches(S, c, "fp8q_rms_norm", 3, 33)
    b = back_args()
    _launches(S, b, "rms_norm_backward", 40, 64)
    _launches(S, lambda: b(dh=None), "rms_norm_backward", 40, 64)
    _launches(S, lambda: b(dx=b.addr("dy")), "rms_norm_backward", 40, 64)
    _launches(S, lambda: b(dx=b.addr("dh")), "rms_norm_backward", 40, 64)
    _launches(S, lambda: b(rows=0, dy=None, h=None, w=None, rstd=None, dh=None, dx=None, ws=None, wsb=0),
              "rms_norm_backward", 0, 64)
    ids, s, p, o = Buf(8 * 60), Buf(4 * 60), Buf(4 * 60), Buf(4 * 9)
    for w, name in ((4, "moe_sort32"), (8, "moe_sort64")):
        _launches(S, lambda: S.fp8q_moe_sort(P(ids.addr), w, 10, 6, 8, P(s.addr), P(p.addr), P(o.addr), None,
                                             0, None), name, 60, 8)
    _launches(S, lambda: S.fp8q_moe_sort(None, 4, 0, 6, 8, None, None, P(o.addr), None, 0, None),
              "moe_sort32", 0, 8)
    x, sl, d = Buf(10 * 30), Buf(4 * 60), Buf(60 * 30)
    _launches(S, lambda: S.fp8q_moe_permute(P(x.addr), 30, None, 0, P(sl.addr), 10, 6, 60, P(d.addr), None,
                                            None), "moe_permute", 10, 30)
    rows, sc, out = Buf(60 * 64 * 2), Buf(60 * 4), Buf(10 * 64 * 4)
    for f, scales in ((0, None), (1, sc), (2, sc), (3, sc)):
        _launches(S, lambda: S.fp8q_moe_combine(P(rows.addr), f, scales and P(scales.addr), P(sl.addr), None,
                                                10, 6, 60, 64, P(out.addr), 0, None), "moe_combine", 10, 64)
    _launches(S, lambda: S.fp8q_moe_combine(None, 0, None, P(sl.addr), None, 10, 6, 0, 64, P(out.addr), 1, None),
              "moe_combine", 10, 64)
    dy, dr, w, dw = Buf(10 * 64 * 2), Buf(60 * 64 * 2), Buf(4 * 60), Buf(4 * 60)
    _launches(S, lambda: S.fp8q_moe_combine_backward(P(dy.addr), P(rows.addr), P(sl.addr), P(w.addr), 10, 6, 60,
                                                     64, P(dr.addr), P(dw.addr), None),
              "moe_combine_backward", 10, 64)


# The Python functions' refusals that need no GPU.

def test_binding_refuses_what_is_no_gpu_tensor_of_the_right_type():
    bf, f32, i32 = (torch.zeros(2, 64, dtype=d) for d in (torch.bfloat16, torch.float32, torch.int32))
    w = torch.ones(64)
    for call in (lambda: fq.fp8q_rms_norm_quantize(bf, w), lambda: fq.mx8_rms_norm_quantize(bf, w),
                 lambda: fq.fp8q_rms_norm_backward(bf, bf, w, w), lambda: fq.fp8q_moe_sort(i32, 4),
                 lambda: fq.fp8q_moe_permute(bf, i32), lambda: fq.fp8q_moe_combine(bf, i32),
                 lambda: fq.fp8q_moe_combine_backward(bf, bf, i32, f32)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
    for call in (lambda: fq.fp8q_rms_norm_quantize(f32, w), lambda: fq.mx8_rms_norm_quantize(None, w),
                 lambda: fq.fp8q_rms_norm_backward(f32, bf, w, w), lambda: fq.fp8q_moe_sort(f32, 4),
                 lambda: fq.fp8q_moe_sort([1, 2], 4), lambda: fq.fp8q_moe_permute("x", i32),
                 lambda: fq.fp8q_moe_combine(f32, i32),
                 lambda: fq.fp8q_moe_combine_backward(f32, bf, i32, f32)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        fq.fp8q_moe_combine(bf, i32, out_dtype=torch.float16)


def test_a_flag_without_a_truth_value_is_refused():
    bf, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.ones(64)
    for flag in ("want_h", "want_y", "want_rstd"):
        for norm in (fq.fp8q_rms_norm_quantize, fq.mx8_rms_norm_quantize):
            with pytest.raises(TypeError, match=flag):
                norm(bf, w, **{flag: torch.ones(2)})


def test_missing_libraries_fail_loudly(monkeypatch, tmp_path):
    with pytest.raises(RuntimeError, match="not built"):
        layer.layer_lib(str(tmp_path / "absent.so"))
    monkeypatch.setattr(layer, "_native", None)
    monkeypatch.setattr(layer, "BINDING_PATH", str(tmp_path / "absent.so"))
    with pytest.raises(RuntimeError, match="not built"):
        fq.fp8q_moe_sort(torch.zeros(1, 1, dtype=torch.int32), 4)
