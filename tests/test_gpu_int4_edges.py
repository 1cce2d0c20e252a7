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


@pytest.mark.parametrize("m", [1, 5])
@pytest.mark.parametrize("asym", [False, True])
def test_product_under_the_largest_scales(m, asym):
    """float32 scales up to 3e38 with x small enough for a finite result: within
    the products' bound (test_gpu_int4.py), as for any other scale."""
    torch = need_gpu()
    rows, cols, group = 40, 640, 64
    g = torch.Generator(device="cuda").manual_seed(4)
    packed = torch.randint(0, 256, (rows * cols // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = 3e37 * (1 + 9 * torch.rand((rows, cols // group), generator=g, device="cuda"))
    zeros = torch.randint(0, 16, scales.shape, generator=g, device="cuda", dtype=torch.uint8) if asym else None
    x = (torch.randn((m, cols), generator=g, device="cuda") * 2.0 ** -20).bfloat16()
    W = nf4.Int4Weight(packed, rows, cols, group, scales, zeros)
    q = torch.stack((packed >> 4, packed & 15), 1).reshape(rows, -1, group).double()
    w = ((q - (zeros.double()[..., None] if asym else 8.0)) * scales.double()[..., None]).reshape(rows, cols)
    ref, size = x.double() @ w.t(), x.double().abs() @ scales.double().repeat_interleave(group, 1).t()
    for kind in (torch.float32, torch.bfloat16):
        y = nf4.nf4_int4_gemv(W, x, y_dtype=kind)
        bound = torch.finfo(kind).eps / 2 * ref.abs() + (group + cols / group + 24) * 2.0 ** -24 * 64 * size
        assert ((y.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("m", [2, 5, 16])
@pytest.mark.parametrize("rows,cols,group", [(40, 96, 32), (83, 640, 64), (300, 3584, 128), (70, 8256, 64)])
def test_rows_of_x_stay_apart(m, rows, cols, group):
    """Infinities and NaN in one row of x: NaN in its row of y, every
    other row as without them, bit for bit."""
    torch = need_gpu()
    for asym in (False, True):
        w = torch.randn((rows, cols), device="cuda")
        W = nf4.quantize_int4(w, group=group, symmetric=not asym)
        x = torch.randn((m, cols), device="cuda").bfloat16()
        clean = nf4.nf4_int4_gemv(W, x, y_dtype=torch.float32)
        for row, at, value in ((m - 1, cols - 1, "inf"), (0, cols // 2, "-inf"), (m // 2, 0, "nan")):
            bad = x.clone()
            bad[row, at] = float(value)
            got = nf4.nf4_int4_gemv(W, bad, y_dtype=torch.float32)
            others = torch.arange(m, device="cuda") != row
            assert torch.equal(got[others], clean[others])
            assert got[row].isnan().all()
