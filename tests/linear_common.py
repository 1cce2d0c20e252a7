"""What the later tests of nf4_linear share: inputs, and the definition in 64 bits
with bounds of one reading of the weight, the one in float32.

A weight enters the products of a few rows of x as its level rounded to fp16
(2^-11 of the weight at most) and the scale in float32, those of more rows as
the fp16 product of level and scale, each rounded to fp16 (3 2^-11).  Sums of K
products in float32: K 2^-24 of the sum of magnitudes.  The adapters' thin factor
is carried as two bf16 parts: 2^-16.  The activation's slope is at most 1.13, its
own evaluation good to 2^-16 of the result.  Then one rounding to bf16."""

from __future__ import annotations

import dequant_matmul_nf4_amd as nf4
from tests.layer_common import F32, HALF, SLOPE_MOST, act64, worst

LEVELS, PRODUCTS = 2.0 ** -11, 3 * 2.0 ** -11


def weight(torch, rows, cols, scales="int8", fp4=False):
    w = (torch.randn((rows, cols), device="cuda") / cols ** 0.5).bfloat16()
    return nf4.quantize_weight(w, double_quant=scales != "plain", dq_type="fp8" if scales == "fp8" else "int8",
                               quant_type="fp4" if fp4 else "nf4")


def inputs(torch, m, rows, cols, bias=None, residual=False, rank=0):
    x = torch.randn((m, cols), device="cuda").bfloat16()
    kw = {}
    if bias:
        kw["bias"] = (0.5 * torch.randn(rows, device="cuda")).to(torch.float32 if bias == "f32" else torch.bfloat16)
    if residual:
        kw["residual"] = torch.randn((m, rows), device="cuda").bfloat16()
    if rank:
        kw |= dict(lora_a=(torch.randn((rank, cols), device="cuda") / cols ** 0.5).bfloat16(),
                   lora_b=(torch.randn((rows, rank), device="cuda") * 0.3).bfloat16(), lora_scale=2.0)
    return x, kw


def product64(torch, W, x, kw, rounding):
    """z of nf4_linear(W, x, **kw) in float64, and how far the sums may be from it."""
    wd, xd = nf4.nf4_dequantize(W, out_dtype=torch.float32).double(), x.double().reshape(-1, W.cols)
    terms = W.cols + 8
    z = xd @ wd.t()
    err = (terms * F32 + rounding) * (xd.abs() @ wd.abs().t())
    if kw.get("lora_a") is not None:
        a, b, s = kw["lora_a"].double(), kw["lora_b"].double(), kw["lora_scale"]
        z = z + s * (xd @ a.t()) @ b.t()
        err = err + (2.0 ** -16 + (terms + a.shape[0]) * F32) * abs(s) * (xd.abs() @ a.abs().t()) @ b.abs().t()
    if kw.get("bias") is not None:
        z = z + kw["bias"].double()
    return z, err + 4 * F32 * z.abs()


def share_of_bound(torch, W, x, kw, y, rounding, pre=None):
    """The largest share of its bound that an element of y (and pre) is off."""
    z, err = product64(torch, W, x, kw, rounding)
    v = act64(torch, kw.get("act", "none"), z)
    out = v + kw["residual"].double().reshape(z.shape) if kw.get("residual") is not None else v
    off = SLOPE_MOST * err + 2.0 ** -16 * v.abs() + 1e-35
    share = worst((y.double() - out).abs(), HALF["bf16"] * (out.abs() + off) + off)
    if pre is not None:
        share = max(share, worst((pre.double() - z).abs(), HALF["bf16"] * (z.abs() + err) + err + 1e-35))
    return share
