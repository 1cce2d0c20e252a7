"""Slopes in the negative tails, relative to themselves: dbias of a single row is
the slope in float32, so nothing of it is hidden by a rounding to bf16.

With u = 2^-24, the hardware's exponential and reciprocal good to 2 u and every
operation of float32 to u, relative errors for z <= -2 (z of 8 bits, so z^2 is
exact) are, with the loss where the slope's two terms cancel:
  silu       s (1 + z (1 - s)): the exponent's argument |z| log2(e) loses 1.5 u of its
             size (constant and product), 1.5 |z| u of s; s another 5 u, the products
             and the difference 4 u; the terms cancel by (1 + |z|) / (|z| - 1) <= 3:
             (4.5 |z| + 27) u
  gelu       exp(-z^2 / 2): .75 z^2 u and 2 u; the polynomial 1.2e-7 of itself (2 u) and
             7 u as evaluated, t and the products 5 u, the density's factor 1.5 u; the
             terms cancel by 1.6: (1.2 z^2 + 26) u
  gelu_tanh  the argument a = 2 sqrt(2 / pi) |z| (1 + .044715 z^2) from 5 roundings and
             log2(e): 6.5 u of a; s another 5 u, its factor 6 u; cancelling by 1.6:
             (10.4 a + 18) u
and anything below 2^-118 may be flushed to zero (the exponential or its reciprocal
below 2^-126 times a factor of up to 2^8)."""

from __future__ import annotations

import math

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.layer_common import slope64, worst

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
FLUSHED = 2.0 ** -118


def allowed(act, z):
    if act == "silu":
        return (4.5 * z.abs() + 27) * U
    if act == "gelu":
        return (1.2 * z * z + 26) * U
    return (10.4 * 2 * math.sqrt(2 / math.pi) * z.abs() * (1 + 0.044715 * z * z) + 18) * U


def tail(torch):
    """Every bf16 from -2 to -120."""
    bits = torch.arange(0xC000, 0xC2F1, device="cuda", dtype=torch.int32).to(torch.int16)
    z = bits.view(torch.bfloat16)
    assert float(z[0]) == -2 and float(z[-1]) == -120
    return z.reshape(1, -1)


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_of_the_negative_tail(act):
    torch = need_gpu()
    z = tail(torch)
    _, slope = nf4.nf4_act_backward(torch.ones_like(z), z, act)
    ref = slope64(torch, act, z.double())[0]
    off = allowed(act, z.double()[0]) * ref.abs() + FLUSHED
    share = worst((slope.double() - ref).abs(), off)
    say("slope tail", act, share)
    assert share <= 1.0, (act, share)
    # where the slope is not flushed it is far from nothing and of the right sign
    seen = ref.abs() > 2 * FLUSHED
    assert int(seen.sum()) > 150 and (slope[seen] < 0).all()


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_round_once(act):
    """dz is that slope, rounded once."""
    torch = need_gpu()
    z = tail(torch)
    dz, slope = nf4.nf4_act_backward(torch.ones_like(z), z, act)
    assert torch.equal(dz[0], slope.bfloat16())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_of_the_negative_tail(act):
    """y of nf4_linear where z is the bias alone: relative to the definition, within its rounding to bf16 and
    what the slope's tail is allowed (its own exponential, no cancellation)."""
    torch = need_gpu()
    from tests.layer_common import HALF, act64
    z = tail(torch)[0]
    rows = z.numel()
    W = nf4.NF4Weight(torch.full((rows * 32,), 0x77, dtype=torch.uint8, device="cuda"), rows, 64,
                      absmax=torch.ones(rows, device="cuda"))
    for m in (1, 5, 600):
        x = torch.zeros((m, 64), dtype=torch.bfloat16, device="cuda")
        y, pre = nf4.nf4_linear(W, x, bias=z.float(), act=act, save_pre=True)
        assert torch.equal(pre[m - 1], z)
        ref = act64(torch, act, z.double())
        off = allowed(act, z.double()) * ref.abs() + FLUSHED
        share = worst((y[m - 1].double() - ref).abs(), HALF["bf16"] * (ref.abs() + off) + off)
        assert share <= 1.0, (act, m, share)
        seen = ref.abs() > 2 * FLUSHED
        assert (y[m - 1][seen] < 0).all()
