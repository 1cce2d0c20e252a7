"""Host-only checks of the calls around the products (no GPU needed): bad
arguments are refused before the device is touched, by the C ABI and by the
binding."""

from __future__ import annotations

import ctypes
import math
import os

import pytest

import dequant_matmul_nf4_amd as nf4

A, B, C, WS = 0x10000, 0x20000, 0x30000, 1 << 30  # aligned addresses that nothing dereferences


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(nf4.LIB_PATH):
        from dequant_matmul_nf4_amd import build
        build.build()
    return nf4.lib()


def _w(**kw):
    base = dict(packed=A, rows=32, cols=64, blocksize=64, absmax=B, blocksize2=256)
    base.update(kw)
    return ctypes.byref(nf4.nf4_weight(**base))


def _ep(**kw):
    return ctypes.byref(nf4.nf4_epilogue(**kw))


def _lin(L, w=None, x=A, m=4, y=B, ep=None, la=None, lb=None, r=0, s=1.0, ws=None, wsn=0):
    return L.nf4_linear(w or _w(), x, m, y, ep, la, lb, r, s, ws, wsn, None)


def _actb(L, dy=A, pre=B, m=4, rows=32, act=2, dz=C, db=A, ws=None, wsn=0):
    return L.nf4_act_backward(dy, pre, m, rows, act, dz, db, ws, wsn, None)


def _bal(L, x=A, t=0, ids=A, mask=None, tokens=10, experts=8, slots=2, coef=0.1, loss=A, counts=A, mean=A, ws=A, wsn=WS):
    return L.nf4_expert_balance(x, t, ids, mask, tokens, experts, slots, coef, loss, counts, mean, ws, wsn, None)


def _balb(L, x=A, t=0, counts=A, mask=None, tokens=10, experts=8, slots=2, coef=0.1, dloss=None, out=B):
    return L.nf4_expert_balance_backward(x, t, counts, mask, tokens, experts, slots, coef, dloss, out, None)


def _g(*entries):
    return (nf4.nf4_grad * len(entries))(*[nf4.nf4_grad(*e) for e in entries])


def _norm(L, g=None, count=1, norm=A, ws=A, wsn=WS):
    g = g if g is not None else _g((A, None, 10, 0, 0))
    return L.nf4_grad_norm(g if g else None, count, norm, ws, wsn, None)


def _clip(L, g=None, count=1, most=1.0, total=None, norm=A, ws=A, wsn=WS):
    g = g if g is not None else _g((A, B, 10, 0, 0))
    return L.nf4_grad_clip(g if g else None, count, most, total, norm, ws, wsn, None)


N, S, AL, D, W = nf4.NF4_ERR_NULL, nf4.NF4_ERR_SIZE, nf4.NF4_ERR_ALIGN, nf4.NF4_ERR_DTYPE, nf4.NF4_ERR_WORKSPACE
CASES = [("linear", _lin, kw, code) for kw, code in [
    (dict(w=_w(packed=None)), N), (dict(x=None), N), (dict(y=None), N), (dict(w=_w(cols=96)), S), (dict(w=_w(cols=1 << 23)), S),
    (dict(m=0), S), (dict(m=(1 << 31) + 1), S), (dict(x=A + 8), AL), (dict(y=B + 2), AL), (dict(x=B), AL), (dict(la=A), N), (dict(lb=A), N),
    (dict(r=4), S), (dict(la=A, lb=A, r=0), S), (dict(la=A, lb=A, r=65), S), (dict(la=A, lb=A, r=4, s=math.inf), S),
    (dict(la=A + 2, lb=A, r=4, ws=A, wsn=WS), AL), (dict(la=A, lb=A, r=4), W), (dict(la=A, lb=A, r=4, ws=A, wsn=8), W),
    (dict(la=A, lb=A, r=4, ws=A + 16, wsn=WS), AL), (dict(ep=_ep(act=5)), D), (dict(ep=_ep(act=-1)), D),
    (dict(ep=_ep(bias=A, bias_dtype=2)), D), (dict(ep=_ep(bias=A + 2, bias_dtype=0)), AL), (dict(ep=_ep(bias=A + 1, bias_dtype=1)), AL),
    (dict(ep=_ep(residual=A + 8)), AL), (dict(ep=_ep(pre=A + 2)), AL), (dict(ep=_ep(pre=B)), AL), (dict(ep=_ep(pre=C, residual=C)), AL),
    (dict(w=_w(quant_type=3)), D), (dict(w=_w(blocksize=32)), nf4.NF4_ERR_BLOCKSIZE)]]
CASES += [("act backward", _actb, kw, code) for kw, code in [
    (dict(dy=None), N), (dict(pre=None), N), (dict(dz=None, db=None), N), (dict(m=0), S), (dict(rows=0), S), (dict(rows=1 << 31), S),
    (dict(m=1 << 31, rows=1 << 20), S), (dict(act=9), D), (dict(dy=A + 2), AL), (dict(pre=A + 8), AL), (dict(dz=A + 4), AL),
    (dict(dz=B), AL), (dict(db=A + 2), AL), (dict(m=1 << 20), W), (dict(m=1 << 20, ws=A, wsn=4), W), (dict(m=1 << 20, ws=A + 2, wsn=WS), AL)]]
CASES += [("balance", _bal, kw, code) for kw, code in [
    (dict(x=None), N), (dict(ids=None), N), (dict(loss=None), N), (dict(counts=None), N), (dict(mean=None), N), (dict(t=3), D),
    (dict(tokens=0), S), (dict(tokens=1 << 31), S), (dict(tokens=1 << 30, slots=2), S), (dict(experts=0), S), (dict(experts=1025), S),
    (dict(slots=0), S), (dict(coef=math.nan), S), (dict(x=A + 2), AL), (dict(x=A + 1, t=1), AL), (dict(ids=A + 2), AL), (dict(loss=A + 2), AL),
    (dict(ws=None), W), (dict(wsn=16), W), (dict(ws=A + 4), AL)]]
CASES += [("balance backward", _balb, kw, code) for kw, code in [
    (dict(x=None), N), (dict(counts=None), N), (dict(out=None), N), (dict(t=-1), D), (dict(tokens=0), S), (dict(experts=2000), S),
    (dict(slots=0), S), (dict(coef=math.inf), S), (dict(out=B + 2), AL), (dict(counts=A + 2), AL), (dict(dloss=A + 2), AL)]]
CASES += [("norm", _norm, kw, code) for kw, code in [
    (dict(norm=None), N), (dict(norm=A + 2), AL), (dict(count=-1), S), (dict(count=(1 << 20) + 1), S), (dict(g=(), count=2), N),
    (dict(g=_g((None, None, 5, 0, 0))), N), (dict(g=_g((A, None, -1, 0, 0))), S), (dict(g=_g((A, None, 1 << 40, 0, 0))), S),
    (dict(g=_g((A, None, 5, 3, 0))), D), (dict(g=_g((A + 2, None, 5, 0, 0))), AL), (dict(g=_g((A + 1, None, 5, 1, 0))), AL),
    (dict(ws=None), W), (dict(wsn=64), W), (dict(ws=A + 4), AL)]]
CASES += [("clip", _clip, kw, code) for kw, code in [
    (dict(most=-1.0), S), (dict(most=math.nan), S), (dict(most=math.inf), S), (dict(norm=A + 2), AL), (dict(total=A + 2), AL),
    (dict(g=_g((A, None, 5, 0, 0))), N), (dict(g=_g((A, B, 5, 0, 7))), D), (dict(g=_g((A, B + 2, 5, 0, 0))), AL),
    (dict(g=_g((A, A, 5, 0, 1))), D), (dict(count=1 << 21), S), (dict(g=_g((A, B, 5, 0, 0), (A, B, -5, 0, 0)), count=2), S)]]


@pytest.mark.parametrize("i", range(len(CASES)), ids=[f"{c[0]} {i}" for i, c in enumerate(CASES)])
def test_refused_on_the_host(L, i):
    name, call, kw, code = CASES[i]
    rc = call(L, **kw)
    assert rc == code, (name, kw, rc, nf4.nf4_last_error())
    assert nf4.nf4_last_error().startswith("nf4_")


def test_workspaces(L):
    assert nf4.nf4_linear_workspace(0, 32, 64, 4) == 0 and nf4.nf4_linear_workspace(8, 32, 64, 65) == 0
    assert nf4.nf4_linear_workspace(1, 32, 64, 4) > 0
    assert nf4.nf4_act_backward_workspace(0, 5) == 0 and nf4.nf4_act_backward_workspace(1, 5) == 0
    # at most 256 rows of sums, whatever m
    assert 0 < nf4.nf4_act_backward_workspace(1 << 25, 1000) <= 256 * 1000 * 4
    assert nf4.nf4_expert_balance_workspace(0, 8) == 0 and nf4.nf4_expert_balance_workspace(8, 1025) == 0
    assert 0 < nf4.nf4_expert_balance_workspace((1 << 31) - 1, 1024) < 4 << 20
    assert nf4.nf4_grad_workspace(-1) == 0 and 0 < nf4.nf4_grad_workspace(0) <= nf4.nf4_grad_workspace(100000)


def test_struct_layout():
    assert ctypes.sizeof(nf4.nf4_epilogue) == 32 and nf4.nf4_epilogue.residual.offset == 16
    assert ctypes.sizeof(nf4.nf4_grad) == 32 and nf4.nf4_grad.dtype.offset == 24


def test_binding_refuses():
    torch = pytest.importorskip("torch")
    bf = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = nf4.NF4Weight(torch.zeros(2048, dtype=torch.uint8), 64, 64, absmax=torch.ones(64))
    with pytest.raises(ValueError):
        nf4.nf4_linear(w, bf)                                   # host tensors
    with pytest.raises(ValueError):
        nf4.nf4_act_backward(bf, bf, "tanh")
    with pytest.raises(ValueError):
        nf4.nf4_act_backward(bf, bf, "silu")
    x, ids = torch.zeros((6, 8)), torch.zeros((6, 2), dtype=torch.int32)
    for call in (lambda: nf4.nf4_expert_balance(x, ids, 2, 0.1), lambda: nf4.nf4_expert_balance(x[0], ids, 2, 0.1),
                 lambda: nf4.nf4_expert_balance(x, ids, 0, 0.1), lambda: nf4.nf4_expert_balance(torch.zeros((6, 1025)), ids, 2, 0.1),
                 lambda: nf4.nf4_expert_balance_backward(x, ids, 2, 0.1), lambda: nf4.nf4_grad_norm([]), lambda: nf4.nf4_grad_norm([x]),
                 lambda: nf4.nf4_grad_clip([x], 1.0), lambda: nf4.nf4_grad_clip([], 1.0)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        nf4.nf4_expert_balance(x.double(), ids, 2, 0.1)
    with pytest.raises(TypeError):
        nf4.nf4_grad_norm([ids])
