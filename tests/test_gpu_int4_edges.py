"""int4 weights at the ends of their types: infinite values, the largest scales,
rows of x that are not finite.  The definitions and the numpy forms are those of
test_gpu_int4.py."""

from __future__ import annotations

import numpy as np
import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.test_gpu_int4 import _pack, _quantize_np, _types

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(22)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("asym", [False, True])
def test_infinite_values_under_a_saturated_scale(kind, group, asym):
    """A float16 scale saturates, so an infinite value has a quotient, and its
    code is the end of the range on its side; groups without one are as ever."""
    torch = need_gpu()
    say("int4 infinite", kind, group, asym)
    rows, cols = 6, 256
    w = np.random.default_rng(6).standard_normal((rows, cols)).astype(np.float32)
    w[0, 3] = np.inf
    w[1, 5] = -np.inf
    w[2, [0, group - 1]] = np.inf, -np.inf
    w[3, cols - 1], w[3, cols - 2] = np.inf, 3.0e4
    w[4, :group] = -np.inf
    t = torch.from_numpy(w).to(_types(torch)[kind])
    W = nf4.quantize_int4(t.cuda(), group=group, symmetric=not asym, scale_dtype=torch.float16)
    q, s, z = _quantize_np(t.float().numpy(), group, asym, "f16")
    assert np.array_equal(W.scales.float().cpu().numpy(), s)
    assert s[0, 0] == 65504 and s[5, 0] < 1
    if asym:
        assert np.array_equal(W.zeros.cpu().numpy(), z)
    else:
        codes = q[[0, 1, 2, 2, 3], [3, 5, 0, group - 1, cols - 1]]
        assert codes.tolist() == [15, 0, 15, 0, 15]
    assert np.array_equal(W.packed.cpu().numpy(), _pack(q))
