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
