"""Refusals of the binding's expert calls that need no GPU."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4


@pytest.mark.parametrize("change", [
    dict(),                                       # dweights is wanted, and needs y
    dict(want=("dy",), dweights=True),            # given, and needs y
    dict(want=("dy",), dy=(12 * 64,)),            # the buffer's rows are m
    dict(want=("dy",), slots=5),                  # positions do not fill tokens
    dict(want=("dy",), slots=0),
    dict(want=("dy",), y=(12 * 64,)),
    dict(want=("dy",)),                           # host tensors
])
def test_combine_backward_refuses(change):
    torch = pytest.importorskip("torch")

    def bf16(shape):
        return torch.zeros(shape, dtype=torch.bfloat16)

    kw = dict(change)
    dout, position, slots = bf16((6, 64)), torch.zeros((6, 2), dtype=torch.int32), kw.pop("slots", 2)
    y = bf16(kw.pop("y")) if "y" in kw else None
    if "dy" in kw:
        kw["dy"] = bf16(kw["dy"])
    if "dweights" in kw:
        kw["dweights"] = torch.zeros(6, 2)
    with pytest.raises(ValueError):
        nf4.nf4_expert_combine_backward(dout, y, position, slots, **kw)


def test_batches_of_no_token_are_checked():
    torch = pytest.importorskip("torch")
    none = torch.empty((0, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        nf4.nf4_expert_plan(none, 4)                                    # host tensors
    with pytest.raises(ValueError):
        nf4.nf4_expert_combine(torch.empty((0, 64), dtype=torch.bfloat16), none, 2)
    with pytest.raises(ValueError):
        nf4.nf4_expert_combine(torch.empty((0,), dtype=torch.bfloat16), none, 2)
