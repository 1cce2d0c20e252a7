"""Host-only checks of the expert and int4 calls (no GPU needed): bad arguments
are refused before the device is touched, by the C ABI and by the binding."""

from __future__ import annotations

import ctypes
import os

import pytest

import dequant_matmul_nf4_amd as nf4

A, B, WS = 0x10000, 0x20000, 1 << 20  # aligned addresses that nothing dereferences


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


def _i4(**kw):
    base = dict(packed=A, rows=16, cols=128, group=64, scale_dtype=nf4.NF4_F16, scales=B, zeros=None)
    base.update(kw)
    return ctypes.byref(nf4.nf4_int4_weight(**base))


def _plan(L, ids=A, n=10, experts=4, order=A, position=A, offsets=A, ws=None, wsn=0):
    return L.nf4_expert_plan(ids, n, experts, order, position, offsets, ws, wsn, None)


def _gemm(L, w=None, experts=4, x=A, x_rows=10, index=None, slots=1, offsets=A, m=10, y=A):
    return L.nf4_expert_gemm(w or _w(), experts, x, x_rows, index, slots, offsets, m, y, None)


def _dx(L, w=None, experts=4, dy=A, offsets=A, m=10, dx=A):
    return L.nf4_expert_gemm_dx(w or _w(), experts, dy, offsets, m, dx, None)


def _comb(L, y=A, m=10, position=A, tokens=5, slots=2, cols=64, weights=None, out=A):
    return L.nf4_expert_combine(y, m, position, tokens, slots, cols, weights, out, None)


def _cb(L, dout=A, y=A, m=10, position=A, tokens=5, slots=2, cols=64, weights=None, dy=A, dw=A):
    return L.nf4_expert_combine_backward(dout, y, m, position, tokens, slots, cols, weights, dy, dw, None)


N, S, AL, D, W, B_ = (nf4.NF4_ERR_NULL, nf4.NF4_ERR_SIZE, nf4.NF4_ERR_ALIGN, nf4.NF4_ERR_DTYPE, nf4.NF4_ERR_WORKSPACE,
                      nf4.NF4_ERR_BLOCKSIZE)
CASES = [
    ("plan", _plan, dict(ids=None), N), ("plan", _plan, dict(order=None), N), ("plan", _plan, dict(position=None), N),
    ("plan", _plan, dict(offsets=None), N), ("plan", _plan, dict(n=0), S), ("plan", _plan, dict(n=1 << 31), S),
    ("plan", _plan, dict(experts=0), S), ("plan", _plan, dict(experts=1025), S), ("plan", _plan, dict(ids=A + 2), AL),
    ("plan", _plan, dict(n=100000), W), ("plan", _plan, dict(n=100000, ws=A, wsn=16), W),
    ("plan", _plan, dict(n=100000, ws=A + 2, wsn=WS), AL),
    ("gemm", _gemm, dict(w=_w(packed=None)), N), ("gemm", _gemm, dict(x=None), N), ("gemm", _gemm, dict(y=None), N),
    ("gemm", _gemm, dict(offsets=None), N), ("gemm", _gemm, dict(experts=0), S), ("gemm", _gemm, dict(experts=2000), S),
    ("gemm", _gemm, dict(experts=5), S), ("gemm", _gemm, dict(w=_w(cols=96)), S), ("gemm", _gemm, dict(w=_w(cols=1 << 23)), S),
    ("gemm", _gemm, dict(m=0), S), ("gemm", _gemm, dict(m=1 << 31), S), ("gemm", _gemm, dict(x_rows=0), S),
    ("gemm", _gemm, dict(x_rows=9), S), ("gemm", _gemm, dict(index=A, slots=0), S), ("gemm", _gemm, dict(x=A + 8), AL),
    ("gemm", _gemm, dict(y=A + 2), AL), ("gemm", _gemm, dict(offsets=A + 1), AL), ("gemm", _gemm, dict(index=A + 2), AL),
    ("gemm", _gemm, dict(w=_w(quant_type=3)), D), ("gemm", _gemm, dict(w=_w(blocksize=128)), B_),
    ("dx", _dx, dict(dy=None), N), ("dx", _dx, dict(dx=None), N), ("dx", _dx, dict(offsets=None), N),
    ("dx", _dx, dict(w=_w(rows=36), experts=4), S), ("dx", _dx, dict(experts=3), S), ("dx", _dx, dict(m=0), S),
    ("dx", _dx, dict(w=_w(rows=1 << 24), experts=1), S), ("dx", _dx, dict(dy=A + 4), AL), ("dx", _dx, dict(dx=A + 4), AL),
    ("combine", _comb, dict(y=None), N), ("combine", _comb, dict(position=None), N), ("combine", _comb, dict(out=None), N),
    ("combine", _comb, dict(cols=12), S), ("combine", _comb, dict(cols=0), S), ("combine", _comb, dict(tokens=0), S),
    ("combine", _comb, dict(slots=0), S), ("combine", _comb, dict(tokens=1 << 30, slots=2), S), ("combine", _comb, dict(m=0), S),
    ("combine", _comb, dict(y=A + 2), AL), ("combine", _comb, dict(weights=A + 2), AL),
    ("combine backward", _cb, dict(dout=None), N), ("combine backward", _cb, dict(position=None), N),
    ("combine backward", _cb, dict(dy=None, dw=None), N), ("combine backward", _cb, dict(y=None), N),
    ("combine backward", _cb, dict(cols=4), S), ("combine backward", _cb, dict(dy=A + 2), AL),
    ("combine backward", _cb, dict(dw=A + 2), AL),
    ("int4 gemv", lambda L, w=None, x=A, xt=1, m=1, y=A, yt=1: L.nf4_int4_gemv(w or _i4(), x, xt, m, y, yt, None), dict(x=None), N),
]
CASES += [("int4 gemv", CASES[-1][1], kw, code) for kw, code in [
    (dict(y=None), N), (dict(m=0), S), (dict(m=17), S), (dict(xt=0), D), (dict(xt=7), D), (dict(yt=3), D), (dict(x=A + 8), AL),
    (dict(w=_i4(packed=None)), N), (dict(w=_i4(scales=None)), N), (dict(w=_i4(group=48)), B_), (dict(w=_i4(group=256, cols=256)), B_),
    (dict(w=_i4(cols=96)), S), (dict(w=_i4(cols=0)), S), (dict(w=_i4(rows=0)), S), (dict(w=_i4(rows=1 << 40)), S),
    (dict(w=_i4(scale_dtype=5)), D), (dict(w=_i4(packed=A + 8)), AL), (dict(w=_i4(scales=B + 1)), AL),
    (dict(w=_i4(scales=B + 2, scale_dtype=nf4.NF4_F32)), AL)]]
CASES += [("int4 quantize", lambda L, w=None, x=A, t=0: L.nf4_int4_quantize(x, t, w or _i4(), None), kw, code) for kw, code in [
    (dict(x=None), N), (dict(t=3), D), (dict(x=A + 4), AL), (dict(w=_i4(cols=32)), S)]]
CASES += [("int4 dequantize", lambda L, w=None, o=A, t=0: L.nf4_int4_dequantize(w or _i4(), o, t, None), kw, code) for kw, code in [
    (dict(o=None), N), (dict(t=-1), D), (dict(o=A + 4), AL), (dict(w=_i4(group=0)), B_)]]


@pytest.mark.parametrize("i", range(len(CASES)), ids=[f"{c[0]} {i}" for i, c in enumerate(CASES)])
def test_refused_on_the_host(L, i):
    name, call, kw, code = CASES[i]
    rc = call(L, **kw)
    assert rc == code, (name, kw, rc, nf4.nf4_last_error())
    assert nf4.nf4_last_error().startswith("nf4_")
    # a NULL weight descriptor of each call that takes one
    assert L.nf4_int4_gemv(None, A, 1, 1, A, 1, None) == N and L.nf4_expert_gemm(None, 1, A, 1, None, 1, A, 1, A, None) == N


def test_plan_workspace(L):
    assert nf4.nf4_expert_plan_workspace(0, 4) == 0 and nf4.nf4_expert_plan_workspace(10, 0) == 0
    assert nf4.nf4_expert_plan_workspace(1 << 31, 4) == 0 and nf4.nf4_expert_plan_workspace(10, 1025) == 0
    # at most 256 rows of counts, whatever n
    assert 0 < nf4.nf4_expert_plan_workspace((1 << 31) - 1, 1024) <= 256 * 1024 * 4


def test_struct_layout():
    assert ctypes.sizeof(nf4.nf4_int4_weight) == 48
    assert nf4.nf4_int4_weight.group.offset == 24 and nf4.nf4_int4_weight.scales.offset == 32


def test_binding_refuses_host_tensors_and_shapes():
    torch = pytest.importorskip("torch")
    ids = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):
        nf4.nf4_expert_plan(ids, 4)
    with pytest.raises(ValueError):
        nf4.quantize_int4(torch.zeros(4, 100), group=64)
    with pytest.raises(ValueError):
        nf4.quantize_int4(torch.zeros(128), group=64)
    w = nf4.Int4Weight(torch.zeros(128, dtype=torch.uint8), 4, 64, 64, torch.ones(4, 1))
    with pytest.raises(ValueError):
        nf4.nf4_int4_gemv(w, torch.zeros(1, 64, dtype=torch.bfloat16))
    for bad in (dict(group=16), dict(cols=96), dict(rows=0)):
        with pytest.raises(ValueError):
            nf4.Int4Weight(**{**dict(packed=w.packed, rows=4, cols=64, group=64, scales=w.scales), **bad}).check()
    with pytest.raises(TypeError):
        nf4.Int4Weight(w.packed, 4, 64, 64, torch.ones(4, 1, dtype=torch.float64)).check()
    with pytest.raises(ValueError):
        nf4.nf4_expert_combine(torch.zeros(4, 64, dtype=torch.bfloat16), ids, 3)
    with pytest.raises(ValueError):
        nf4.nf4_expert_gemm_dx(nf4.NF4Weight(w.packed, 4, 64, absmax=torch.ones(4)), 3, torch.zeros(1, 64), ids)
