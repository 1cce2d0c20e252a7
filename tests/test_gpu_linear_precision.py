"""How near nf4_linear comes to the weight itself: less than half as far as its
rounding to bf16 would be.

A result in bf16 hides that, so the residual takes the exact product, rounded to
bf16, away: what is left is at most 2^-8 of it, and the result's own rounding 2^-16
(1.5e-5 of the product).  Then, for random x, the error's norm over the norm of the
products with the weight's rounding to bf16 is that of the weights' root mean squares:
  bf16        a step of 2^-7 over sqrt(12) for a value of [1, 2): 2.26e-3, at least
              1.13e-3 of the value
  levels      each off by 2^-11 at most, 4.9e-4: 0.43 of that at most
  products    two more roundings, 2^-10 over sqrt(12) each: 6.3e-4 of the value in all
              at most, where the value is a power of two and bf16's 2.26e-3; for evenly
              spread values 2.26e-3 / 1.53 = 1.48e-3 against (4.9e-4, 1.85e-4, 1.85e-4)
              5.6e-4: 0.38
so 0.5 of it; weights in bf16 are at 1."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.layer_common import HALF, worst
from tests.linear_common import LEVELS, PRODUCTS, inputs, product64, weight

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(61)


# one and two rows of wide or many rows; decode batches, and more rows with little work; these meet the levels
FEW = [(1, 1003, 4160), (2, 1003, 4160), (1, 12301, 704), (1, 4096, 4096), (5, 1000, 64), (16, 333, 576), (3, 40, 14400), (16, 4096, 4096),
       (64, 512, 512), (300, 100, 320), (150, 2001, 4160)]
# cut reductions and whole tiles: level times scale
MANY = [(96, 4096, 14336), (330, 2001, 4160), (300, 9007, 640), (2100, 4100, 192), (1030, 4352, 256), (2048, 4096, 1024)]


def check(torch, W, x, kw, rounding, label):
    z, err = product64(torch, W, x, kw, rounding)
    res = -z.bfloat16()
    y = nf4.nf4_linear(W, x, residual=res, **kw)
    left = z + res.double()
    off = (y.double() - left).abs()
    share = worst(off, err + HALF["bf16"] * (left.abs() + err) + 1e-35)
    wd = nf4.nf4_dequantize(W, out_dtype=torch.float32).double()
    rounded = x.double() @ (wd.bfloat16().double() - wd).t()
    part = float(off.norm() / rounded.norm())
    say("linear precision", label, f"of the bound {share:.3f}, of bf16's error {part:.3f}")
    assert share <= 1.0, (label, share)
    assert part <= 0.5, (label, part)


@pytest.mark.parametrize("scales,fp4", [("int8", False), ("fp8", False), ("plain", False), ("int8", True), ("plain", True)])
@pytest.mark.parametrize("m,rows,cols", FEW)
def test_few_rows_meet_the_levels(m, rows, cols, scales, fp4):
    torch = need_gpu()
    W = weight(torch, rows, cols, scales, fp4)
    x, kw = inputs(torch, m, rows, cols, "f32")
    check(torch, W, x, kw, LEVELS, (m, rows, cols, scales, fp4))


@pytest.mark.parametrize("scales,fp4", [("int8", False), ("fp8", False), ("plain", False), ("int8", True), ("plain", True)])
@pytest.mark.parametrize("m,rows,cols", MANY)
def test_many_rows_meet_level_times_scale(m, rows, cols, scales, fp4):
    torch = need_gpu()
    W = weight(torch, rows, cols, scales, fp4)
    x, kw = inputs(torch, m, rows, cols, "f32")
    check(torch, W, x, kw, PRODUCTS, (m, rows, cols, scales, fp4))


@pytest.mark.parametrize("m,rows,cols", [(1, 1003, 4160), (2, 1003, 4160), (16, 333, 576), (330, 2001, 4160), (1030, 4352, 256)])
@pytest.mark.parametrize("up,down", [(60, -50), (-60, 50), (90, -100), (-100, 90)])
def test_of_any_magnitude(m, rows, cols, up, down):
    torch = need_gpu()
    W = nf4.quantize_weight(torch.randn((rows, cols), device="cuda").bfloat16() * 2.0 ** up)
    x = (torch.randn((m, cols), device="cuda") * 2.0 ** down).bfloat16()
    check(torch, W, x, {}, LEVELS if m <= 16 else PRODUCTS, (m, rows, cols, up, down))


@pytest.mark.parametrize("rank", [1, 16, 48])
@pytest.mark.parametrize("m,rows,cols", [(1, 1003, 4160), (2, 1003, 4160), (16, 333, 576), (330, 2001, 4160), (1030, 4352, 256), (700, 33, 1088)])
def test_adapters_add_no_more(m, rows, cols, rank):
    """Their thin factor in two bf16 parts: 2^-16 of their share, within the same half of the weight's rounding."""
    torch = need_gpu()
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, rank=rank)
    check(torch, W, x, kw, LEVELS if m <= 16 or rows == 33 else PRODUCTS, (m, rows, cols, rank))
