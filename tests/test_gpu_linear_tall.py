"""nf4_linear over weights of many rows (vocabulary projections) with one, two and
three rows of x, on both sides of 65536 weight rows, where a workgroup's partial
sums of two rows of x are full."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.linear_common import LEVELS, PRODUCTS, inputs, share_of_bound, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(53)


@pytest.mark.parametrize("scales", ["int8", "fp8", "plain"])
@pytest.mark.parametrize("rank", [0, 5])
@pytest.mark.parametrize("rows,cols", [(65536, 128), (65537, 128), (70001, 128), (65537, 2112), (131075, 4096), (128256, 4096), (66000, 8256)])
def test_tall_weights(rows, cols, rank, scales):
    torch = need_gpu()
    W = weight(torch, rows, cols, scales)
    for m in (1, 2, 3):
        say("linear tall", m, rows, cols, rank, scales)
        x, kw = inputs(torch, m, rows, cols, "f32", residual=True, rank=rank)
        y, pre = nf4.nf4_linear(W, x, act="silu", save_pre=True, **kw)
        share = share_of_bound(torch, W, x, dict(kw, act="silu"), y, LEVELS, pre)
        assert share <= 1.0, (m, share)
        assert torch.equal(y, nf4.nf4_linear(W, x, act="silu", **kw))


@pytest.mark.parametrize("rows,cols", [(65537, 128), (128256, 4096)])
def test_tall_weight_in_a_graph(rows, cols):
    """Two rows of x captured once and replayed with others, eager work between."""
    torch = need_gpu()
    say("linear tall graph", rows, cols)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, 2, rows, cols, "bf16")
    y = torch.empty((2, rows), dtype=torch.bfloat16, device="cuda")
    nf4.nf4_linear(W, x, y=y, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        nf4.nf4_linear(W, x, y=y, **kw)
    for rep in range(3):
        x.copy_(torch.randn_like(x))
        want = nf4.nf4_linear(W, x, **kw)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), rep
        share = share_of_bound(torch, W, x, kw, y, LEVELS)
        assert share <= 1.0, share


def test_weight_past_32_bits():
    """2^32 weights and more: rows of y at both ends and past the 2^32nd weight, for each kernel's number of rows of x."""
    torch = need_gpu()
    rows, cols = 140000, 32768
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    nb = rows * cols // 64
    packed = torch.randint(0, 256, (rows * cols // 2,), generator=g, device="cuda", dtype=torch.uint8)
    W = nf4.NF4Weight(packed, rows, cols, qabsmax=torch.randint(-127, 128, (nb,), generator=g, device="cuda", dtype=torch.int8),
                      absmax2=0.01 + 0.01 * torch.rand(-(-nb // 256), generator=g, device="cuda"), mean=torch.full((1,), 0.03, device="cuda"))
    picked = (0, 65536, 131071, 131072, 139488)  # blocks of 512 rows, of whole groups of scales
    for m in (1, 2, 5, 40, 300, 700):
        say("linear past 32 bits", m)
        x, kw = inputs(torch, m, rows, cols, "f32")
        y = nf4.nf4_linear(W, x, act="silu", **kw)
        for first in picked:
            lo, n = first * cols, 512 * cols
            part = nf4.NF4Weight(packed[lo // 2:(lo + n) // 2], 512, cols, qabsmax=W.qabsmax[lo // 64:(lo + n) // 64],
                                 absmax2=W.absmax2[lo // 16384:(lo + n) // 16384], mean=W.mean)
            some = dict(bias=kw["bias"][first:first + 512], act="silu")
            share = share_of_bound(torch, part, x, some, y[:, first:first + 512], LEVELS if m <= 5 else PRODUCTS)
            assert share <= 1.0, (m, first, share)


def test_outputs_past_32_bits():
    """2^31 outputs and more: rows of y at both ends, y and pre."""
    torch = need_gpu()
    m, rows, cols = 33000, 65600, 64
    say("linear outputs past 32 bits")
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16")
    y, pre = nf4.nf4_linear(W, x, act="relu", save_pre=True, **kw)
    for t in (0, 16384, 32700, 32999):
        share = share_of_bound(torch, W, x[t:t + 1], dict(kw, act="relu"), y[t:t + 1], PRODUCTS, pre[t:t + 1])
        assert share <= 1.0, (t, share)
