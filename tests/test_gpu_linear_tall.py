"""nf4_linear over weights of many rows (vocabulary projections) with one, two and
three rows of x, on both sides of 65536 weight rows, where a workgroup's partial
sums of two rows of x are full."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.linear_common import LEVELS, inputs, share_of_bound, weight

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
