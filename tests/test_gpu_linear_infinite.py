"""Rows of x with an infinity through nf4_linear: the definition's infinities, of its
signs, and its NaN (an infinity times a weight of zero) in that row and nothing in
any other, wherever the infinity lies, the last columns of a row above all, which the
kernels read again where a row ends inside what they take at a time."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.linear_common import inputs, weight

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(59)


def same_class(torch, got, want):
    """NaN in the same places, infinities of the same signs, everything else finite."""
    w = torch.where(want.abs() > 3.4e38, want * INF, want)
    return (torch.equal(got.isnan(), w.isnan()) and torch.equal(got == INF, w == INF)
            and torch.equal(got == -INF, w == -INF))


# one and two rows over one segment and several; a decode batch over both; cut reductions, whole
# tiles; widths that end inside what a wave takes and whole ones
ROW = [(1, 300, 4160), (2, 300, 4160), (1, 301, 2112), (2, 301, 2112), (1, 12301, 704), (2, 12301, 704), (1, 100, 8192), (2, 33, 14400)]
FEW = [(3, 100, 64), (7, 100, 192), (16, 333, 576), (5, 40, 1088), (9, 300, 4416), (3, 17, 14400), (16, 64, 1024), (40, 70, 320), (2, 33, 576), (40, 9001, 4416), (150, 2001, 4160),
       (97, 8199, 2112)]
MID = [(330, 2001, 4160), (300, 9007, 640), (520, 4001, 2112), (200, 14343, 256)]
TILES = [(1030, 4352, 256), (2100, 4100, 192), (700, 9007, 640)]


@pytest.mark.parametrize("scales", ["int8", "fp8", "plain"])
@pytest.mark.parametrize("m,rows,cols", ROW + FEW + MID + TILES)
def test_infinity_anywhere_in_a_row(m, rows, cols, scales):
    torch = need_gpu()
    say("linear infinite", m, rows, cols, scales)
    W = weight(torch, rows, cols, scales)
    x, kw = inputs(torch, m, rows, cols, "f32", residual=True)
    clean = nf4.nf4_linear(W, x, **kw)
    wd = nf4.nf4_dequantize(W, out_dtype=torch.float32).double()
    t = m // 2
    keep = torch.arange(m, device="cuda") != t
    for places in ((cols - 1,), (cols - 8,), (cols - 33,), (cols - 64,), (0,), (cols // 2,), (cols - 1, cols - 2)):
        for sign in (1.0, -1.0):
            bad = x.clone()
            for p in places:
                bad[t, p] = sign * INF
            y, pre = nf4.nf4_linear(W, bad, save_pre=True, **kw)
            want = torch.zeros(rows, dtype=torch.float64, device="cuda")
            for p in places:  # finite terms change nothing beside an infinity
                want = want + bad[t, p].double() * wd[:, p]
            assert same_class(torch, y[t].double(), want), (places, sign, int(y[t].isnan().sum()), int(want.isnan().sum()))
            assert same_class(torch, pre[t].double(), want), (places, sign, "pre")
            assert torch.equal(y[keep], clean[keep]), (places, sign, "other rows")


@pytest.mark.parametrize("m,rows,cols", [(1, 300, 4160), (2, 301, 2112), (7, 100, 192), (16, 333, 576), (150, 2001, 4160),
                                         (1030, 4352, 256)])
def test_row_of_nan(m, rows, cols):
    """A NaN makes its whole row NaN and touches no other."""
    torch = need_gpu()
    say("linear nan", m, rows, cols)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16")
    clean = nf4.nf4_linear(W, x, **kw)
    for p in (0, cols - 1):
        bad = x.clone()
        bad[m - 1, p] = float("nan")
        y = nf4.nf4_linear(W, bad, **kw)
        assert y[m - 1].isnan().all() and torch.equal(y[:m - 1], clean[:m - 1])


@pytest.mark.parametrize("rank", [1, 3, 17])
@pytest.mark.parametrize("m,rows,cols", [(1, 300, 4160), (2, 301, 2112), (7, 100, 192), (16, 333, 576), (150, 2001, 4160), (330, 2001, 4160),
                                         (700, 9007, 640), (1030, 4352, 256), (700, 33, 1088)])
def test_infinity_through_adapters(m, rows, cols, rank):
    """The adapters' thin factor of such a row is infinite itself; B decides between its infinities and NaN."""
    torch = need_gpu()
    say("linear infinite adapters", m, rows, cols, rank)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16", rank=rank)
    kw["lora_b"] = kw["lora_b"].abs() + 0.01  # the sum over the rank keeps a sign where all of A's column have one
    kw["lora_a"][:, -1] = kw["lora_a"][:, -1].abs() + 0.01
    clean = nf4.nf4_linear(W, x, **kw)
    wd = nf4.nf4_dequantize(W, out_dtype=torch.float32).double()
    t = m - 1 if m < 3 else m // 3
    keep = torch.arange(m, device="cuda") != t
    seen = 0
    for place in (cols - 1, 5):
        for sign in (1.0, -1.0):
            bad = x.clone()
            bad[t, place] = sign * INF
            y, pre = nf4.nf4_linear(W, bad, save_pre=True, **kw)
            thin = bad[t, place].double() * kw["lora_a"][:, place].double()
            want = bad[t, place].double() * wd[:, place] + (thin * kw["lora_b"].double()).sum(1)
            assert same_class(torch, y[t].double(), want), (place, sign, int(y[t].isnan().sum()), int(want.isnan().sum()))
            assert same_class(torch, pre[t].double(), want), (place, sign, "pre")
            assert torch.equal(y[keep], clean[keep])
            seen += int(want.isinf().sum())
    assert seen > 0
