"""The C ABI of include/fp8q_model.h: the library exports what the header
declares, and rejects every bad request on the host before any launch; the
Python functions refuse tensors that do not fit.

As in test_layer_abi.py, the validation tests never reach a launch, and are
skipped where a GPU is visible; tests/test_model_abi_sanitized.py runs this
file against a host-check build, where accepted calls can run too.
"""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import dequantize_reduce_transfer_amd as fq
from dequantize_reduce_transfer_amd import build, model
from test_layer_abi import ERR_ALIGN, ERR_ARG, ERR_NULL, ERR_OVERLAP, OK, Buf, P, no_gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fp8q_model.h")
LIB = os.environ.get("FP8Q_MODEL_HOSTCHECK", model.LIB_PATH)


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(model.LIB_PATH):
        build.build_model()
    if not os.path.exists(model.BINDING_PATH):
        build.build_model_binding()


def L():
    return model.model_lib(LIB)


def _declared():
    return sorted(re.findall(r"^FP8Q_API\s+\w+\s+(\w+)\s*\(", open(HEADER).read(), re.M))


def test_header_declares_the_abi():
    assert _declared() == sorted(model.EXPORTS)
    text = open(HEADER).read()
    assert re.search(r"#define FP8Q_EXPERTS_MAX_PAIRS %d\b" % model.EXPERTS_MAX_PAIRS, text)
    assert re.search(r"#define FP8Q_EXPERTS_MAX_SIZE %d\b" % model.EXPERTS_MAX_SIZE, text)


def test_library_exports_exactly_what_is_declared():
    out = subprocess.run(["nm", "-D", "--defined-only", model.LIB_PATH], capture_output=True, text=True).stdout
    assert {line.split()[-1] for line in out.splitlines() if " T " in line} == set(_declared())


def test_header_compiles_as_c():
    source = ('#include "fp8q_model.h"\nint main(void) { fp8q_grad g = {0}; fp8q_expert_matrix m = {0}; '
              'return g.count == 0 && m.rows == 0 && sizeof g == %d ? 0 : 1; }\n' % ctypes.sizeof(model.Grad))
    r = subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", "-pedantic", "-fsyntax-only", "-I",
                        os.path.join(ROOT, "include"), "-x", "c", "-"], input=source, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def caller(function, order, bufs, **values):
    """function(**change): a call with good arguments, some of them changed."""
    args = dict({k: P(b.addr) for k, b in bufs.items()}, **values)

    def call(**change):
        a = dict(args, **change)
        return getattr(L(), function)(*[a[k] for k in order], None)
    call.addr = lambda k, off=0: P(bufs[k].addr + off)
    return call


def route_call():
    bufs = dict(l=Buf(4 * 12 * 16), w=Buf(4 * 12 * 4), ids=Buf(4 * 12 * 4))
    return caller("fp8q_moe_route", ["l", "dt", "tokens", "experts", "topk", "norm", "w", "ids"], bufs, dt=0,
                  tokens=12, experts=16, topk=4, norm=1)


def route_backward_call():
    bufs = dict(dw=Buf(4 * 12 * 4), l=Buf(4 * 12 * 16), w=Buf(4 * 12 * 4), ids=Buf(4 * 12 * 4), dl=Buf(4 * 12 * 16))
    return caller("fp8q_moe_route_backward",
                  ["dw", "l", "dt", "w", "ids", "tokens", "experts", "topk", "norm", "dl"], bufs, dt=0, tokens=12,
                  experts=16, topk=4, norm=0)


@no_gpu
def test_route_validation():
    for c, out in ((route_call(), "w"), (route_backward_call(), "dl")):
        for bad in (dict(dt=2), dict(dt=-1), dict(experts=0), dict(experts=1025), dict(topk=0), dict(topk=17),
                    dict(experts=1024, topk=65), dict(tokens=1 << 40)):
            assert c(**bad) == ERR_ARG, bad
        assert c(tokens=0) == OK and c(tokens=0, l=None, ids=None) == OK
        for k in ("l", "w", "ids", out):
            assert c(**{k: None}) == ERR_NULL, k
        for k in ("l", *(["dl"] if out == "dl" else [])):
            assert c(**{k: c.addr(k, 8)}) == ERR_ALIGN, k
        for k in ("w", "ids"):
            assert c(**{k: c.addr(k, 2)}) == ERR_ALIGN, k
    c = route_call()
    for k, at in (("w", c.addr("ids")), ("w", c.addr("l", 4)), ("ids", c.addr("l", 4 * 12 * 16 - 4))):
        assert c(**{k: at}) == ERR_OVERLAP, k
    c = route_backward_call()
    for at in (c.addr("l", 16), c.addr("w"), c.addr("ids"), c.addr("dw")):
        assert c(dl=at) == ERR_OVERLAP


E, I, H, T, K = 5, 64, 96, 6, 2
EXPERTS_ORDER = ["x", "ids", "id_bytes", "w", "format", "gate", "up", "down", "tokens", "topk", "experts", "hidden",
                 "inter", "out", "dt", "ws", "ws_bytes"]


def experts_call(fmt=3):
    rows, per = {0: (2, None), 1: (1, 4), 2: (1, 4), 3: (1, 32)}[fmt]
    scales = None if per is None else Buf(4 * E * max(I, H) * 4)
    data = {k: Buf(rows * 2 * E * I * H) for k in ("gate", "up", "down")}
    bufs = dict(x=Buf(2 * T * H), ids=Buf(8 * T * K), w=Buf(4 * T * K), out=Buf(4 * T * H), ws=Buf(6 * T * K * I))
    call = caller("fp8q_moe_experts", EXPERTS_ORDER, bufs, id_bytes=4, format=fmt, tokens=T, topk=K, experts=E,
                  hidden=H, inter=I, dt=0, ws_bytes=6 * T * K * I,
                  **{k: ctypes.byref(call_matrix(data[k], scales, H if k == "down" else I)) for k in data})
    call.matrix = lambda k, **change: ctypes.byref(call_matrix(data[k], scales, **dict(dict(expert_rows=H if k == "down" else I), **change)))
    call.data, call.scales = data, scales
    return call


def call_matrix(data, held, expert_rows, **change):
    m = model.ExpertMatrix(data.addr, held.addr if held else None, expert_rows)
    for k, v in change.items():
        setattr(m, k, v)
    return m


@no_gpu
@pytest.mark.parametrize("fmt", range(4))
def test_experts_validation(fmt):
    c = experts_call(fmt)
    for bad in (dict(format=4), dict(format=-1), dict(id_bytes=2), dict(dt=2), dict(topk=0), dict(topk=65),
                dict(tokens=513), dict(experts=0), dict(experts=1025), dict(hidden=65536 + 32),
                dict(inter=65536 + 32), dict(ws_bytes=6 * T * K * I - 1),
                dict(gate=c.matrix("gate", expert_rows=I - 1)), dict(down=c.matrix("down", expert_rows=H - 1)),
                dict(up=c.matrix("up", expert_rows=1 << 40)),
                *([dict(hidden=48), dict(inter=48)] if fmt == 3 else []),
                *([dict(gate=c.matrix("gate", scales=c.addr("x").value))] if fmt == 0 else [])):
        assert c(**bad) == ERR_ARG, bad
    assert c(tokens=0) == OK and c(hidden=0) == OK and c(tokens=0, gate=None) == OK
    for k in ("x", "ids", "w", "gate", "up", "down", "out", "ws"):
        assert c(**{k: None}) == ERR_NULL, k
    assert c(gate=c.matrix("gate", rows=None)) == ERR_NULL
    if fmt:
        assert c(down=c.matrix("down", scales=None)) == ERR_NULL
    for k in ("x", "out", "ws"):
        assert c(**{k: c.addr(k, 8)}) == ERR_ALIGN, k
    assert c(ids=c.addr("ids", 2)) == ERR_ALIGN and c(ids=c.addr("ids", 4), id_bytes=8) == ERR_ALIGN
    assert c(w=c.addr("w", 2)) == ERR_ALIGN
    if fmt == 0:
        assert c(gate=c.matrix("gate", rows=c.data["gate"].addr + 1)) == ERR_ALIGN
    if fmt in (1, 2):
        assert c(up=c.matrix("up", scales=c.scales.addr + 2)) == ERR_ALIGN
    for k, at in (("out", c.addr("x")), ("out", c.addr("ws", 16)), ("ws", c.addr("x", 16)), ("out", c.addr("w")),
                  ("ws", c.addr("ids"))):
        assert c(**{k: at}) == ERR_OVERLAP, k
    for k in ("gate", "up", "down"):
        assert c(out=P(c.data[k].addr + 16)) == ERR_OVERLAP
        assert c(ws=P(c.data[k].addr + 16)) == ERR_OVERLAP
    if fmt:
        assert c(out=P(c.scales.addr)) == ERR_OVERLAP


def grads(*entries):
    """A struct array of (buffer or address, scales or None, count, scale count, dtype)."""
    a = (model.Grad * max(1, len(entries)))()
    for i, (d, s, n, sn, t) in enumerate(entries):
        a[i] = model.Grad(d if not isinstance(d, Buf) else d.addr, s if not isinstance(s, Buf) else s.addr, n, sn, t)
    return a


@no_gpu
def test_grad_validation():
    a, b, q, s, one = Buf(4000), Buf(2000), Buf(1000), Buf(32), Buf(16)
    total, norm, ws = Buf(8), Buf(4), Buf(1 << 16)
    good = [(a, None, 1000, 0, 0), (b, None, 1000, 0, 1), (q, s, 1000, 8, 2), (q, one, 1000, 1, 3)]

    def both(entries, out=None, sumsq=None, n=None):
        g, n = grads(*entries), len(entries) if n is None else n
        return (L().fp8q_grad_sumsq(g, n, out or P(total.addr), P(ws.addr), 1 << 16, None),
                L().fp8q_grad_clip(g, n, sumsq or P(total.addr), 1.0, 1e-6, out or P(norm.addr), None))

    for bad, want in ((good + [(a, None, 1, 0, 4)], ERR_ARG), (good + [(a, None, 1, 0, -1)], ERR_ARG),
                      ([(a, s, 1000, 8, 0)], ERR_ARG), ([(b, None, 1000, 1, 1)], ERR_ARG),
                      ([(q, s, 1000, 7, 2)], ERR_ARG), ([(q, s, 1000, 0, 3)], ERR_ARG),
                      ([(a, None, (1 << 40) + 1, 0, 0)], ERR_ARG), ([(None, None, 5, 0, 0)], ERR_NULL),
                      ([(q, None, 1000, 8, 2)], ERR_NULL), ([(a.addr + 2, None, 5, 0, 0)], ERR_ALIGN),
                      ([(b.addr + 1, None, 5, 0, 1)], ERR_ALIGN), ([(q, s.addr + 2, 100, 1, 2)], ERR_ALIGN)):
        assert both(bad) == (want, want), bad
    assert L().fp8q_grad_sumsq(None, 2, P(total.addr), P(ws.addr), 1 << 16, None) == ERR_NULL
    assert L().fp8q_grad_clip(None, 2, P(total.addr), 1.0, 1e-6, P(norm.addr), None) == ERR_NULL
    g = grads(*good)
    assert L().fp8q_grad_sumsq(g, 4, None, P(ws.addr), 1 << 16, None) == ERR_NULL
    assert L().fp8q_grad_sumsq(g, 4, P(total.addr + 4), P(ws.addr), 1 << 16, None) == ERR_ALIGN
    assert L().fp8q_grad_sumsq(g, 4, P(total.addr), P(ws.addr + 8), 1 << 15, None) == ERR_ALIGN
    many = Buf(1 << 20)                      # a list that needs a workspace
    large = grads((many, None, 1 << 18, 0, 0), *good)
    assert L().fp8q_grad_sumsq(large, 5, P(total.addr), P(ws.addr), 7, None) == ERR_ARG
    assert L().fp8q_grad_sumsq(large, 5, P(total.addr), None, 1 << 16, None) == ERR_NULL
    for at in (a.addr + 8, b.addr, q.addr, s.addr + 8, one.addr, many.addr + 4096, ws.addr):
        assert L().fp8q_grad_sumsq(large, 5, P(at // 8 * 8), P(ws.addr), 1 << 16, None) == ERR_OVERLAP
    for at in (a.addr, many.addr + 4096):
        assert L().fp8q_grad_sumsq(large, 5, P(total.addr), P(at), 1 << 16, None) == ERR_OVERLAP
    for bad in (dict(m=-1.0), dict(m=float("nan")), dict(e=-1.0), dict(e=float("nan")), dict(e=float("inf"))):
        assert L().fp8q_grad_clip(g, 4, P(total.addr), bad.get("m", 1.0), bad.get("e", 1e-6), P(norm.addr),
                                  None) == ERR_ARG, bad
    assert L().fp8q_grad_clip(g, 4, None, 1.0, 1e-6, P(norm.addr), None) == ERR_NULL
    assert L().fp8q_grad_clip(g, 4, P(total.addr), 1.0, 1e-6, None, None) == ERR_NULL
    assert L().fp8q_grad_clip(g, 4, P(total.addr + 4), 1.0, 1e-6, P(norm.addr), None) == ERR_ALIGN
    assert L().fp8q_grad_clip(g, 4, P(total.addr), 1.0, 1e-6, P(norm.addr + 2), None) == ERR_ALIGN
    for at in (a.addr, b.addr + 1996, s.addr, one.addr, total.addr):
        assert L().fp8q_grad_clip(g, 4, P(total.addr), 1.0, 1e-6, P(at), None) == ERR_OVERLAP
    # written twice: the same tensor, one inside another, the same scales
    for twice in ([(a, None, 1000, 0, 0)] * 2, [(a, None, 1000, 0, 0), (b, None, 9, 0, 1), (a.addr + 400, None, 9, 0, 1)],
                  [(q, s, 1000, 8, 2), (b, None, 9, 0, 1), (q, s, 100, 1, 2)]):
        assert L().fp8q_grad_clip(grads(*twice), len(twice), P(total.addr), 1.0, 1e-6, P(norm.addr),
                                  None) == ERR_OVERLAP, twice


def test_workspaces():
    small, large = grads((Buf(400), None, 100, 0, 0)), grads((Buf(400), None, 1 << 30, 0, 0))
    if LIB == model.LIB_PATH:
        assert L().fp8q_grad_sumsq_workspace(small, 1) == 0
        assert 0 < L().fp8q_grad_sumsq_workspace(large, 1) <= 16384
        many = grads(*[(Buf(16), None, 2, 0, 0)] * 300)
        assert 0 < L().fp8q_grad_sumsq_workspace(many, 300) <= 16384 * 3
        # h, its rows filled up to 16; and of many pairs their y
        assert L().fp8q_moe_experts_workspace(3, 2, 8, 100, 17, 1) == 2 * 2 * 6 * 32
        assert L().fp8q_moe_experts_workspace(3, 2, 8, 100, 17, 0) == 3 * 2 * 6 * 32
        assert L().fp8q_moe_experts_workspace(300, 2, 8, 100, 17, 0) == 3 * 2 * 600 * 32 + 4 * 600 * 100
        # few workgroups of long rows: several parts
        assert L().fp8q_moe_experts_workspace(300, 2, 8, 1024, 4096, 1) == 2 * 2 * 600 * 4096 + 4 * 4 * 600 * 1024
    assert L().fp8q_grad_sumsq_workspace(grads((None, None, 5, 0, 0)), 1) == 0
    assert L().fp8q_moe_experts_workspace(1025, 1, 8, 64, 64, 0) == 0
    assert L().fp8q_moe_experts_workspace(4, 0, 8, 64, 64, 0) == 0
    assert L().fp8q_moe_experts_workspace(4, 1, 8, 64, 64, 7) == 0


def _stub():
    if "FP8Q_MODEL_HOSTCHECK" not in os.environ:
        pytest.skip("needs the host-check build of the library (FP8Q_MODEL_HOSTCHECK)")
    S = L()
    S.model_stub_calls.restype = ctypes.c_long
    S.model_stub_last.restype = ctypes.c_char_p
    S.model_stub_a.restype = S.model_stub_b.restype = ctypes.c_ulonglong
    return S


def _launches(call, name, a, b):
    S = _stub()
    before = S.model_stub_calls()
    assert call() == OK
    assert S.model_stub_calls() == before + 1
    assert (S.model_stub_last().decode(), S.model_stub_a(), S.model_stub_b()) == (name, a, b)


@no_gpu
def test_accepted_calls_reach_their_launchers():
    _stub()
    for norm in (0, 1):
        for dt in (0, 1):
            _launches(lambda: route_call()(norm=norm, dt=dt), "moe_route", 12, 16)
            _launches(lambda: route_backward_call()(norm=norm, dt=dt), "moe_route_backward", 12, 16)
    c = route_backward_call()
    _launches(lambda: c(dl=c.addr("l")), "moe_route_backward", 12, 16)
    _launches(lambda: c(l=None, norm=1), "moe_route_backward", 12, 16)
    for fmt in range(4):
        c = experts_call(fmt)
        for change in ({}, dict(id_bytes=8), dict(dt=1), dict(tokens=1), dict(gate=c.matrix("gate", expert_rows=2 * I))):
            _launches(lambda: c(**change), "moe_experts", change.get("tokens", T), I)
        _launches(lambda: c(inter=0, ws=None, gate=c.matrix("gate", rows=None)), "moe_experts", T, 0)
    a, b, q, s, one, total, norm = Buf(4000), Buf(2000), Buf(1000), Buf(32), Buf(16), Buf(8), Buf(4)
    ws = Buf(64)
    g = grads((a.addr + 4, None, 999, 0, 0), (b.addr + 2, None, 999, 0, 1), (q.addr + 1, s, 999, 8, 2),
              (q, one, 1000, 1, 3), (None, None, 0, 0, 2))
    _launches(lambda: L().fp8q_grad_sumsq(g, 5, P(total.addr), P(ws.addr), 64, None), "grad_sumsq", 5, 999)
    _launches(lambda: L().fp8q_grad_clip(g, 5, P(total.addr), 1.0, 0.0, P(norm.addr), None), "grad_clip", 5, 999)
    _launches(lambda: L().fp8q_grad_clip(g, 5, P(total.addr), float("inf"), 0.0, P(norm.addr), None), "grad_clip", 5, 999)
    _launches(lambda: L().fp8q_grad_sumsq(None, 0, P(total.addr), None, 0, None), "grad_sumsq", 0, 0)
    _launches(lambda: L().fp8q_grad_clip(None, 0, P(total.addr), 1.0, 0.0, P(norm.addr), None), "grad_clip", 0, 0)


# The Python functions' refusals that need no GPU.

def test_binding_refuses_what_is_no_gpu_tensor_of_the_right_type():
    bf, f32, i32 = (torch.zeros(2, 64, dtype=d) for d in (torch.bfloat16, torch.float32, torch.int32))
    f64, w3 = torch.zeros(1, dtype=torch.float64), torch.zeros(4, 32, 64, dtype=torch.bfloat16)
    for call in (lambda: fq.fp8q_moe_route(f32, 2), lambda: fq.fp8q_moe_route_backward(f32, bf, f32, i32),
                 lambda: fq.fp8q_moe_experts(bf, i32, f32, w3, w3, w3), lambda: fq.fp8q_grad_sumsq([f32]),
                 lambda: fq.fp8q_grad_clip([f32, bf], f64, 1.0), lambda: fq.fp8q_grad_clip([], f64, 1.0)):
        with pytest.raises(ValueError, match="on a GPU"):
            call()
    for call in (lambda: fq.fp8q_moe_route(i32, 2), lambda: fq.fp8q_moe_route("x", 2),
                 lambda: fq.fp8q_moe_route_backward(bf, bf, f32, i32),
                 lambda: fq.fp8q_moe_experts(f32, i32, f32, w3, w3, w3), lambda: fq.fp8q_grad_sumsq(f32),
                 lambda: fq.fp8q_grad_sumsq([i32]), lambda: fq.fp8q_grad_sumsq([None]),
                 lambda: fq.fp8q_grad_clip(iter([f32]), f64, 1.0), lambda: fq.fp8q_grad_sumsq(None)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError, match="empty"):
        fq.fp8q_grad_sumsq([])
    with pytest.raises(ValueError, match="one entry a gradient"):
        fq.fp8q_grad_sumsq([f32], scales=[])
    with pytest.raises(ValueError):
        fq.fp8q_grad_sumsq([f32], fmt=7)
    with pytest.raises(ValueError):
        fq.fp8q_moe_experts(bf, i32, f32, w3, w3, w3, out_dtype=torch.float16)


def test_missing_libraries_fail_loudly(monkeypatch, tmp_path):
    with pytest.raises(RuntimeError, match="not built"):
        model.model_lib(str(tmp_path / "absent.so"))
    monkeypatch.setattr(model, "_native", None)
    monkeypatch.setattr(model, "BINDING_PATH", str(tmp_path / "absent.so"))
    with pytest.raises(RuntimeError, match="not built"):
        fq.fp8q_moe_route(torch.zeros(1, 4), 2)
