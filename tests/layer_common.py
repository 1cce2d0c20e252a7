"""What the tests of the layer calls share: definitions in 64 bits, written from
the formulas, and bounds on rounding.

A rounding is off by at most half a step of its type relative to the value:
bf16 2^-8, fp16 2^-11, float32 2^-24."""

from __future__ import annotations

import math

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
F32 = 2.0 ** -24
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
SLOPE_MOST = 1.13   # the steepest of the activations: GELU near z = 1.4


def types(torch):
    return {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def act64(torch, kind, z):
    if kind == "none":
        return z
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def slope64(torch, kind, z):
    """The derivative of act64, by its formula."""
    if kind == "none":
        return torch.ones_like(z)
    if kind == "relu":
        return (z > 0).double()
    if kind == "silu":
        s = torch.sigmoid(z)
        return s + z * s * (1 - s)
    if kind == "gelu":
        return torch.special.erfc(-z / math.sqrt(2)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    s = torch.sigmoid(2 * c * (z + 0.044715 * z ** 3))
    return s + z * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * z * z)


def worst(err, bound):
    """The largest share of its bound that an error takes (NaN counts as over)."""
    share = err / bound
    return math.inf if bool(share.isnan().any()) else float(share.max()) if share.numel() else 0.0
