"""The expert products where their loops run long, and what precision they
promise, against float64.

Precision of a product of few rows per expert (at most 40 on the mean): levels
rounded to float16 (off by at most 2^-11 of their value; not the two bfloat16
parts of an earlier kernel that test_gpu_expert.py's introduction has), x taken
exactly, the block scale and the sums in float32, one rounding to bfloat16.  Per
output, with S = sum |x| |w| over K columns: 2^-8 of the value, and (2^-11 + (K + 8) 2^-24) S
(K additions; the scale's, the power of two's and the reference weight's
roundings).  In the mean square the roundings are independent: the error's
square is that of rounding the reference once, plus the level's,
at most (2^-11)^2 / 3 of the value's square; a tenth is left for their product
and for chance (of 1000 outputs and more).  Weights rounded to bfloat16 after
scaling would double the square."""

from __future__ import annotations

import numpy as np
import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.test_gpu_expert import SHAPES, _check, _counts, _reference, _stack

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(24)


def _offsets(torch, off):
    return torch.from_numpy(np.asarray(off).astype(np.int32)).cuda()


def _check_few(torch, y, ref, mag, cols, least=1e-30):
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + (cols + 8) * 2.0 ** -24) * mag + least
    excess = (y.double() - ref).abs() - bound
    assert excess.max().item() <= 0, (excess / bound).max().item()
    if ref.numel() >= 1000 and ref.any():
        once = (ref.bfloat16().double() - ref).square().sum()
        error = (y.double() - ref).square().sum()
        share = (error / (once + 2.0 ** -22 / 3 * ref.square().sum())).item()
        assert share <= 1.1, share


@pytest.mark.parametrize("experts,rows,cols,m", [s for s in SHAPES if s[3] <= 40 * s[0]] + [(8, 1000, 4096, 16), (3, 272, 8256, 50)])
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_few_rows_keep_the_weight_in_float32(experts, rows, cols, m, kind):
    torch = need_gpu()
    say("few rows", experts, rows, cols, m, kind)
    for i, scales in enumerate(("int8", "fp8", "plain")):
        W = _stack(torch, experts, rows, cols, scales, fp4=(m + i) % 2 == 0)
        off = _counts(kind, experts, m)
        x = torch.randn((m, cols), device="cuda").bfloat16()
        y = nf4.nf4_expert_gemm(W, experts, x, _offsets(torch, off))
        ref, mag = _reference(torch, W, experts, x, off)
        _check_few(torch, y, ref, mag, cols)
        assert torch.equal(y, nf4.nf4_expert_gemm(W, experts, x, _offsets(torch, off)))


@pytest.mark.parametrize("cols", [64, 512, 1088, 4160])
def test_few_rows_of_any_magnitude(cols):
    """Rows of x from near float32's least normal to 2^100, a row of zeros, and
    rows whose values differ by powers of two up to 2^28 within a segment: where
    the largest meets a zero level the smallest alone are the result."""
    torch = need_gpu()
    experts, rows = 2, 1024
    W = _stack(torch, experts, rows, cols, "plain")
    W.absmax *= 2.0 ** 20
    W.packed.view(experts * rows, cols // 2)[:, ::32] &= 0x0F
    W.packed.view(experts * rows, cols // 2)[:, ::32] |= 0x70  # the zero level in the first column of each block
    m = 9
    x = torch.randn((m, cols), device="cuda")
    x[0] *= 2.0 ** -120
    x[1] *= 2.0 ** 100
    x[2] = 0
    x[3] *= 2.0 ** -torch.randint(0, 20, (cols,), device="cuda").float()
    x[4] = (x[4].sign() + x[4] / 8) * 2.0 ** -torch.randint(24, 28, (cols,), device="cuda").float()
    x[4, ::64] = 1.0
    x[5] = x[4] * 2.0 ** 90
    x[6] = x[4] * 2.0 ** -60
    x[7, cols // 2:] = 0
    x = x.bfloat16()
    off = [0, 5, m]
    y = nf4.nf4_expert_gemm(W, experts, x, _offsets(torch, off))
    ref, mag = _reference(torch, W, experts, x, off)
    assert ref[4].abs().max() < 2.0 ** -4 * W.absmax.max() and (y[2] == 0).all()
    for i in range(m):  # row by row: the sums of squares would see the largest alone
        _check_few(torch, y[i:i + 1], ref[i:i + 1], mag[i:i + 1], cols, least=0.0)


# The sizes below put full rounds of 256-row tiles on 256 compute units, and
# 128-row tiles, with steps of 64 columns (rows, for the gradient) by the dozen:
# the ring of three code stages is requested again from the fifth step on.

@pytest.mark.parametrize("experts,rows,cols,m", [
    (3, 4096, 320, 4200), (3, 4096, 384, 4200), (3, 4090, 1088, 4300), (2, 8192, 448, 2500), (1, 14336, 4096, 1000),  # 256 rows
    (3, 520, 320, 480), (5, 272, 1088, 800), (2, 2048, 4160, 446), (70, 40, 576, 9000),                              # 128 rows
])
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_gemm_of_long_rows(experts, rows, cols, m, kind):
    """Every row right in each form of the scales, rows of no expert left, the
    same bits again and with gathered rows."""
    torch = need_gpu()
    say("expert gemm of long rows", experts, rows, cols, m, kind)
    off = _counts(kind, experts, m - 2) + 1
    offsets = _offsets(torch, off)
    index = torch.randint(0, 400, (m,), device="cuda", dtype=torch.int32)
    for i, scales in enumerate(("int8", "fp8", "plain")):
        W = _stack(torch, experts, rows, cols, scales, fp4=(m + i) % 2 == 1)
        x = torch.randn((200, cols), device="cuda").bfloat16()
        xs = x[(index // 2).long()]
        y = torch.full((m, rows), 7.0, dtype=torch.bfloat16, device="cuda")
        nf4.nf4_expert_gemm(W, experts, x, offsets, index=index, slots=2, y=y)
        assert (y[0] == 7).all() and (y[m - 1] == 7).all()
        ref, mag = _reference(torch, W, experts, xs, off)
        _check(y[1:m - 1], ref, mag, cols)
        assert torch.equal(y[1:m - 1], nf4.nf4_expert_gemm(W, experts, xs, offsets)[1:m - 1])


def _one_expert(W, experts, e):
    """Expert e of a stack on its own (its blocks begin at a multiple of 256)."""
    rows = W.rows // experts
    n = rows * W.cols
    at, groups = slice(e * n // 64, (e + 1) * n // 64), slice(e * n // 16384, -(-(e + 1) * n // 16384))
    if W.absmax is not None:
        return nf4.NF4Weight(W.packed[e * n // 2:(e + 1) * n // 2], rows, W.cols, absmax=W.absmax[at], quant_type=W.quant_type)
    assert n % 16384 == 0
    return nf4.NF4Weight(W.packed[e * n // 2:(e + 1) * n // 2], rows, W.cols, qabsmax=W.qabsmax[at], absmax2=W.absmax2[groups],
                         mean=W.mean, dq_type=W.dq_type, quant_type=W.quant_type)


@pytest.mark.parametrize("experts,rows,cols,m", [(3, 4096, 1088, 4200), (3, 4096, 320, 540), (2, 2048, 4160, 446), (3, 512, 768, 270)])
def test_long_rows_equal_the_dense_product(experts, rows, cols, m):
    """Tiles of 256, 128 and 64 rows: nf4_gemm on each expert's rows, bit for bit."""
    torch = need_gpu()
    off = _counts("uneven", experts, m)
    x = torch.randn((m, cols), device="cuda").bfloat16()
    for scales in ("int8", "fp8", "plain"):
        W = _stack(torch, experts, rows, cols, scales)
        y = nf4.nf4_expert_gemm(W, experts, x, _offsets(torch, off))
        for e in range(experts):
            if off[e] < off[e + 1]:
                at = slice(off[e], off[e + 1])
                assert torch.equal(y[at], nf4.nf4_gemm(_one_expert(W, experts, e), x[at])), (scales, e)


@pytest.mark.parametrize("experts,rows,cols,m", [
    (3, 328, 4096, 4200), (3, 392, 4096, 4200), (2, 1000, 5120, 3000), (1, 4096, 14336, 1000),  # 256 rows
    (4, 1000, 8128, 600), (16, 328, 4096, 2000),                                              # 128 rows
    (64, 1024, 2048, 1000),                                                                   # 64 rows
])
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_dx_of_long_reductions(experts, rows, cols, m, kind):
    torch = need_gpu()
    say("expert dx of long reductions", experts, rows, cols, m, kind)
    off = _counts(kind, experts, m - 2) + 1
    offsets = _offsets(torch, off)
    for i, scales in enumerate(("int8", "fp8", "plain")):
        W = _stack(torch, experts, rows, cols, scales, fp4=(m + i) % 2 == 1)
        dy = torch.randn((m, rows), device="cuda").bfloat16()
        dx = torch.full((m, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        nf4.nf4_expert_gemm_dx(W, experts, dy, offsets, dx=dx)
        assert (dx[0] == 7).all() and (dx[m - 1] == 7).all()
        ref, mag = _reference(torch, W, experts, dy, off, dx=True)
        _check(dx[1:m - 1], ref, mag, rows)
        assert torch.equal(dx[1:m - 1], nf4.nf4_expert_gemm_dx(W, experts, dy, offsets)[1:m - 1])
