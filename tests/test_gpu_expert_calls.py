"""Forms of the expert calls that the binding takes: what may be left out, and
sizes of none."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu
from tests.test_gpu_expert import _positions, _stack

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(23)


@pytest.mark.parametrize("weighted", [True, False])
def test_combine_backward_without_y(weighted):
    """dy alone does not need y: the same dy, with and without a buffer for it."""
    torch = need_gpu()
    tokens, slots, cols = 9, 3, 72
    pos = _positions(torch, tokens, slots, 0.0)
    y = torch.randn((tokens * slots, cols), device="cuda").bfloat16()
    wt = torch.rand((tokens, slots), device="cuda") if weighted else None
    dout = torch.randn((tokens, cols), device="cuda").bfloat16()
    dy, _ = nf4.nf4_expert_combine_backward(dout, y, pos, slots, wt)
    got, none = nf4.nf4_expert_combine_backward(dout, None, pos, slots, wt, want=("dy",))
    assert none is None and got.shape == y.shape and torch.equal(got, dy)
    # a buffer of more rows than slots; a dropped slot writes nothing
    pos[4, 1] = -1
    more = torch.full((tokens * slots + 5, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    want, _ = nf4.nf4_expert_combine_backward(dout, torch.zeros_like(more), pos, slots, wt, dy=more.clone())
    got, _ = nf4.nf4_expert_combine_backward(dout, None, pos, slots, wt, dy=more, want=("dy",))
    assert got.data_ptr() == more.data_ptr() and torch.equal(got, want)
    with pytest.raises(ValueError):
        nf4.nf4_expert_combine_backward(dout, None, pos, slots, wt)
    with pytest.raises(ValueError):
        nf4.nf4_expert_combine_backward(dout, None, pos, slots, wt, dweights=torch.zeros((tokens, slots), device="cuda"), want=("dy",))
    with pytest.raises(ValueError):
        nf4.nf4_expert_combine_backward(dout, None, pos, slots, wt, dy=more[:, :64].contiguous(), want=("dy",))
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_expert_combine_backward(dout, None, pos, slots, wt, want=())


@pytest.mark.parametrize("side", [False, True])
def test_batches_of_no_token(side):
    """A rank that no token was sent to: every call answers with what has no
    rows, offsets and gradients of nothing as zeros; checks hold all the same."""
    torch = need_gpu()
    experts, rows, cols, slots = 4, 64, 128, 2
    W = _stack(torch, experts, rows, cols)
    stream = torch.cuda.Stream() if side else None
    offsets = torch.full((experts + 1,), 9, dtype=torch.int32, device="cuda")
    x = torch.empty((0, cols), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    ids = torch.empty((0, slots), dtype=torch.int32, device="cuda")
    order, position, got = nf4.nf4_expert_plan(ids, experts, offsets=offsets, stream=stream)
    y = nf4.nf4_expert_gemm(W, experts, x, offsets, index=order, slots=slots, stream=stream)
    y2 = nf4.nf4_expert_gemm(W, experts, x, offsets, stream=stream)
    dx = nf4.nf4_expert_gemm_dx(W, experts, y, offsets, stream=stream)
    out = nf4.nf4_expert_combine(y, position, slots, stream=stream)
    dy, dw = nf4.nf4_expert_combine_backward(out, y, position, slots, stream=stream)
    only, _ = nf4.nf4_expert_combine_backward(out, None, position, slots, want=("dy",), stream=stream)
    torch.cuda.synchronize()
    assert got.data_ptr() == offsets.data_ptr() and (offsets == 0).all()
    shapes = [tuple(t.shape) for t in (order, position, y, y2, dx, out, dy, dw, only)]
    assert shapes == [(0,), (0,), (0, rows), (0, rows), (0, cols), (0, rows), (0, rows), (0, slots), (0, rows)]
    # tokens, but every slot on another rank: nothing to add up
    away = torch.full((3, slots), -1, dtype=torch.int32, device="cuda")
    wt = torch.rand((3, slots), device="cuda")
    out = torch.full((3, rows), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((3, slots), 7.0, device="cuda")
    torch.cuda.synchronize()
    nf4.nf4_expert_combine(y, away, slots, wt, out=out, stream=stream)
    nf4.nf4_expert_combine_backward(out, y, away, slots, wt, dweights=dw, stream=stream)
    torch.cuda.synchronize()
    assert (out == 0).all() and (dw == 0).all()
    with pytest.raises(ValueError):
        nf4.nf4_expert_gemm(W, experts, x, offsets[:-1].contiguous(), stream=stream)
    with pytest.raises(ValueError):
        nf4.nf4_expert_plan(ids, 0, stream=stream)
    with pytest.raises(TypeError):
        nf4.nf4_expert_plan(ids.long(), experts, stream=stream)


def test_a_batch_that_empties_in_a_graph():
    """Calls on no rows are captured like others: the offsets are zero after
    every replay."""
    torch = need_gpu()
    offsets = torch.empty(5, dtype=torch.int32, device="cuda")
    ids = torch.empty((0,), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        nf4.nf4_expert_plan(ids, 4, offsets=offsets)
    for _ in range(3):
        offsets.fill_(9)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert (offsets == 0).all()
