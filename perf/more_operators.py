"""What stands around the 4-bit products in a layer and a training step: cases to
time and to compare, and the operators' plain forms.

Families (a case names its own in "op"):

  linear              z = x . deq(W)^T + s (x . A^T) . B^T + bias;  y = act(z) + residual,
                      and z itself where a backward pass will want it
  act_backward        dz = dy act'(z) and the bias's gradient, the sum of its rows
  balance             the router's balance loss, its counts per expert and mean probabilities
  balance_backward    that loss's gradient for the logits
  grad_clip           the norm over many gradients, and the gradients scaled to a largest norm

With `own` false, run() computes the plain form in 32 bits (64 where 32 lose
what matters); with `own` true it calls the library."""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
LORA_SCALE = 2.0
LARGEST_PRODUCT = 4096 * 14336 * 4096
LARGEST_WEIGHT = 28672 * 8192
LARGEST_ACT = 4096 * 14336
LARGEST_ROUTE = 131072 * 128
LARGEST_GRADS = 200_000_000


def _lib():
    """The library, imported where its calls are made."""
    import dequant_matmul_nf4_amd as nf4
    return nf4


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token through an attention projection with a bias: latency
        dict(name="linear_token", op="linear", m=1, rows=4096, cols=4096, scales="int8", fp4=False, bias="bf16",
             act="none", residual=False, pre=False, rank=0),
        # a decode batch of 16 through a wide projection with an activation
        dict(name="linear_batch16", op="linear", m=16, rows=28672, cols=8192, scales="int8", fp4=False, bias="none",
             act="silu", residual=False, pre=False, rank=0),
        # a chunk of a prompt (or a large decode batch) through the projection back to the residual stream
        dict(name="linear_chunk", op="linear", m=96, rows=4096, cols=14336, scales="int8", fp4=False, bias="bf16",
             act="none", residual=True, pre=False, rank=0),
        # a training step's forward: adapters, bias, activation, and z kept for the backward pass
        dict(name="linear_train", op="linear", m=4096, rows=14336, cols=4096, scales="int8", fp4=False, bias="f32",
             act="gelu_tanh", residual=False, pre=True, rank=16),
        # the backward pass of that activation and bias
        dict(name="act_backward_train", op="act_backward", m=4096, rows=14336, act="gelu_tanh"),
        # a short ragged batch, the activation with the error function, columns of an odd count
        dict(name="act_backward_ragged", op="act_backward", m=333, rows=11007, act="gelu"),
        # the routers of a small batch over few experts: latency
        dict(name="balance_small", op="balance", tokens=256, experts=8, slots=2, logits="f32", masked=0.0, dropped=0.0,
             closed=0.0),
        # long sequences over many experts, padding masked out, some slots dropped
        dict(name="balance_long", op="balance", tokens=131072, experts=128, slots=8, logits="bf16", masked=0.1,
             dropped=0.05, closed=0.0),
        # their backward passes: many experts with some of them closed, and the ordinary batch of a training step
        dict(name="balance_backward_wide", op="balance_backward", tokens=16384, experts=256, slots=8, logits="f32",
             masked=0.1, dropped=0.0, closed=0.1),
        dict(name="balance_backward_step", op="balance_backward", tokens=8192, experts=8, slots=2, logits="bf16",
             masked=0.0, dropped=0.0, closed=0.0),
        # the adapters' gradients of 80 wide layers, clipped into the optimizer's flat buffer
        dict(name="grad_clip_adapters", op="grad_clip", layers=80, hidden=8192, wide=28672, narrow=1024, rank=16,
             grads="f32", clip=True),
        # the norm alone, over a few small tensors of all types: latency
        dict(name="grad_norm_few", op="grad_clip", count=9, least=16, most=70000, grads="mixed", clip=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of(v, n):
    return max(n, v // n * n)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "act_backward", "balance", "balance_backward", "grad_clip"])
    if op == "linear":
        m, cols = _log(rng, 1, 4096), _of(_log(rng, 64, 14336), 64)
        rows = min(_log(rng, 1, 28672), max(1, LARGEST_PRODUCT // (m * cols)), max(1, LARGEST_WEIGHT // cols))
        return dict(op=op, m=m, rows=rows, cols=cols, scales=rng.choice(["int8", "fp8", "plain"]), fp4=rng.random() < 0.25,
                    bias=rng.choice(["none", "bf16", "f32"]), act=rng.choice(ACTS), residual=rng.random() < 0.5,
                    pre=rng.random() < 0.3, rank=rng.choice([0, 0, rng.randint(1, 64)]))
    if op == "act_backward":
        rows = _log(rng, 1, 28672)
        return dict(op=op, m=_log(rng, 1, min(16384, max(1, LARGEST_ACT // rows))), rows=rows, act=rng.choice(ACTS[1:]))
    if op in ("balance", "balance_backward"):
        experts = _log(rng, 2, 512)
        return dict(op=op, tokens=_log(rng, 1, min(262144, LARGEST_ROUTE // experts)), experts=experts,
                    slots=rng.randint(1, min(8, experts // 2)), logits=rng.choice(["bf16", "f16", "f32"]),
                    masked=rng.choice([0.0, 0.1, 0.9]), dropped=rng.choice([0.0, 0.05]), closed=rng.choice([0.0, 0.2]))
    least = _log(rng, 1, 10000)
    most = _log(rng, least, 2_000_000)
    count = _log(rng, 1, max(1, min(1200, LARGEST_GRADS // most)))
    return dict(op=op, count=count, least=least, most=most, grads=rng.choice(["f32", "bf16", "f16", "mixed"]),
                clip=rng.random() < 0.7)


# --------------------------------------------------------------- the inputs

def _nf4_levels():
    """The 16 NF4 levels: normal quantiles at evenly spaced probabilities on
    either side of zero, divided by the outermost."""
    d = 1 - (1 / 30 + 1 / 32) / 2
    low = torch.special.ndtri(torch.linspace(1 - d, 0.5, 8, dtype=torch.float64)[:-1])
    high = torch.special.ndtri(torch.linspace(0.5, d, 9, dtype=torch.float64)[1:])
    q = torch.cat([low, torch.zeros(1, dtype=torch.float64), high])
    return (q / q[-1]).to(torch.float32)


def _fp4_levels():
    m = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64) / 6
    return torch.cat([m, -m]).to(torch.float32)


def _e4m3_ratios():
    """Value / 448 of the 256 E4M3 codes (the two NaN codes, never drawn, as 0)."""
    c = torch.arange(256)
    e, f = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * 2.0 ** (e - 7).double())
    v = torch.where(c >= 128, -v, v)
    v[[127, 255]] = 0
    return v / 448


def _make_weight(case, g, dev):
    """Codes and scales as the quantizer leaves them, of weights that keep the
    size of x's rows."""
    total = case["rows"] * case["cols"]
    nb = -(-total // 64)
    scale = 1.0 / math.sqrt(case["cols"])
    s = dict(packed=torch.randint(0, 256, (total // 2,), generator=g, device=dev, dtype=torch.uint8),
             levels=(_fp4_levels() if case["fp4"] else _nf4_levels()).to(dev))
    absmax = scale * (2.0 + torch.rand(nb, generator=g, device=dev) * 1.5)
    if case["scales"] == "plain":
        s["absmax"] = absmax
        return s
    s["mean"] = absmax.mean().reshape(1)
    s["absmax2"] = scale * (0.5 + 0.5 * torch.rand(-(-nb // 256), generator=g, device=dev))
    if case["scales"] == "int8":
        s["qabsmax"] = torch.randint(-127, 128, (nb,), generator=g, device=dev, dtype=torch.int16).to(torch.int8)
    else:
        q = torch.randint(0, 127, (nb,), generator=g, device=dev, dtype=torch.int16)
        sign = torch.randint(0, 2, (nb,), generator=g, device=dev, dtype=torch.int16) * 128
        s["qabsmax"] = (q + sign).to(torch.uint8)
        s["ratios"] = _e4m3_ratios().to(dev)
    return s


def _grad_sizes(case):
    """The gradients' sizes: of the adapters A and B of seven projections a layer, or
    spread over least .. most."""
    if "layers" in case:
        h, w, n, r = case["hidden"], case["wide"], case["narrow"], case["rank"]
        one = []
        for rows, cols in ((h, h), (n, h), (n, h), (h, h), (w, h), (w, h), (h, w)):
            one += [r * cols, rows * r]
        return one * case["layers"]
    lo, hi = case["least"], case["most"]
    return [int(lo * (hi / lo) ** (i * 0.6180339887 % 1.0)) for i in range(1, case["count"] + 1)]


def _grad_types(case, count):
    if case["grads"] != "mixed":
        return [DTYPES[case["grads"]]] * count
    return [(torch.float32, torch.bfloat16, torch.float16)[i % 3] for i in range(count)]


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 11)
    op = case["op"]
    s = dict(case)

    def normal(shape, dtype, sigma=1.0):
        return (torch.randn(shape, generator=g, device=dev) * sigma).to(dtype)

    if op == "linear":
        m, rows, cols, r = case["m"], case["rows"], case["cols"], case["rank"]
        s |= _make_weight(case, g, dev)
        s["x"] = normal((m, cols), torch.bfloat16)
        s["b"] = normal((rows,), DTYPES[case["bias"]], 0.5) if case["bias"] != "none" else None
        s["r"] = normal((m, rows), torch.bfloat16) if case["residual"] else None
        s["la"] = normal((r, cols), torch.bfloat16, 1.0 / math.sqrt(cols)) if r else None
        s["lb"] = normal((rows, r), torch.bfloat16, 0.3 / math.sqrt(r)) if r else None
    elif op == "act_backward":
        s["dy"] = normal((case["m"], case["rows"]), torch.bfloat16, 0.1)
        s["z"] = normal((case["m"], case["rows"]), torch.bfloat16, 1.5)
    elif op in ("balance", "balance_backward"):
        t, e = case["tokens"], case["experts"]
        logits = normal((t, e), torch.float32) + 0.5 * torch.randn((1, e), generator=g, device=dev)
        ids = logits.topk(case["slots"], dim=1).indices.to(torch.int32)
        if case["closed"]:  # experts that are closed to a token, and tokens that all are closed to
            shut = torch.rand((t, e), generator=g, device=dev) < case["closed"]
            shut |= torch.rand((t, 1), generator=g, device=dev) < 0.01
            logits = torch.where(shut, torch.full_like(logits, -math.inf), logits)
        s["x"] = logits.to(DTYPES[case["logits"]])
        off = torch.rand(ids.shape, generator=g, device=dev) < case["dropped"]
        s["ids"] = torch.where(off, torch.full_like(ids, -1), ids).contiguous()
        s["mask"] = torch.rand((t,), generator=g, device=dev) >= case["masked"] if case["masked"] else None
        if op == "balance_backward":
            s["counts"] = _counts(s)
            # scaled as where gradients have 16 bits, so that the small ones stay in range
            s["dloss"] = 100 * max(1.0, t * (1 - case["masked"])) * (0.5 + torch.rand((1,), generator=g, device=dev))
    else:
        sizes = _grad_sizes(case)
        sigma = (0.2 + torch.rand(len(sizes), generator=g, device=dev)).tolist()
        types = _grad_types(case, len(sizes))
        s["g"] = [normal((n,), t, v) for n, t, v in zip(sizes, types, sigma)]
        # into one flat buffer of the first gradient's type
        s["flat"] = torch.zeros(sum(sizes), dtype=types[0], device=dev) if case["clip"] else None
        s["max_norm"] = 0.25 * math.sqrt(sum(sizes)) * 0.5
    return s


# ----------------------------------------------------------- the operators

COEF = 0.01


def run(s):
    if own:
        return _run_own(s)
    return PLAIN[s["op"]](s)


def _run_own(s):
    lib = _lib()
    op = s["op"]
    if op == "linear":
        w = lib.NF4Weight(s["packed"], s["rows"], s["cols"], absmax=s.get("absmax"), qabsmax=s.get("qabsmax"),
                          absmax2=s.get("absmax2"), mean=s.get("mean"), dq_type=int(s["scales"] == "fp8"),
                          quant_type=int(s["fp4"]))
        return lib.nf4_linear(w, s["x"], bias=s["b"], act=s["act"], residual=s["r"], lora_a=s["la"], lora_b=s["lb"],
                              lora_scale=LORA_SCALE, save_pre=s["pre"])
    if op == "act_backward":
        return lib.nf4_act_backward(s["dy"], s["z"], s["act"])
    if op == "balance":
        return lib.nf4_expert_balance(s["x"], s["ids"], s["slots"], COEF, mask=s["mask"])
    if op == "balance_backward":
        return lib.nf4_expert_balance_backward(s["x"], s["counts"], s["slots"], COEF, mask=s["mask"], dloss=s["dloss"])
    if not s["clip"]:
        return lib.nf4_grad_norm(s["g"])
    return lib.nf4_grad_clip(s["g"], s["max_norm"], out=s["flat"])


def _unpack(packed):
    """Element 2j is the high half of byte j, element 2j + 1 the low half."""
    return torch.stack((packed >> 4, packed & 15), dim=-1).reshape(-1)


def _dequantized(s):
    if "absmax" in s:
        a = s["absmax"]
    else:
        r = s["qabsmax"].float() / 127 if s["qabsmax"].dtype == torch.int8 else s["ratios"].float()[s["qabsmax"].long()]
        a = r * s["absmax2"].repeat_interleave(256)[:r.numel()] + s["mean"]
    v = s["levels"][_unpack(s["packed"]).to(torch.int32)].reshape(-1, 64)
    return (v * a[:, None]).reshape(s["rows"], s["cols"])


def _act(kind, z):
    if kind == "none":
        return z
    if kind == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def _act_slope(kind, z):
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if kind == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)


def _linear(s):
    x = s["x"].float()
    z = torch.matmul(x, _dequantized(s).t())
    if s["la"] is not None:
        z = z + LORA_SCALE * torch.matmul(torch.matmul(x, s["la"].float().t()), s["lb"].float().t())
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _act(s["act"], z)
    if s["r"] is not None:
        y = y + s["r"].float()
    y = y.to(torch.bfloat16)
    return (y, z.to(torch.bfloat16)) if s["pre"] else y


def _act_backward(s):
    dz = s["dy"].float() * _act_slope(s["act"], s["z"].float())
    return dz.to(torch.bfloat16), dz.sum(0)


def _counts(s):
    """Slots of the kept tokens by expert, then the number of kept tokens."""
    e, ids = s["experts"], s["ids"].long()
    kept = s["mask"][:, None] if s["mask"] is not None else torch.ones_like(ids[:, :1], dtype=torch.bool)
    live = (ids >= 0) & (ids < e) & kept
    key = torch.where(live, ids, torch.full_like(ids, e)).reshape(-1)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    counts[e] = kept.sum()
    return counts.to(torch.int32)


def _probs(s):
    """The routers' probabilities in float32: zeros in rows that are closed altogether, or masked."""
    x = s["x"].float()
    top = x.amax(1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    return p * s["mask"][:, None] if s["mask"] is not None else p


def _balance(s):
    counts, e = _counts(s), s["experts"]
    kept = counts[e].double()
    some = torch.where(kept > 0, kept, torch.ones_like(kept))
    mean = _probs(s).double().sum(0) / some
    loss = COEF * e * (counts[:e].double() / (some * s["slots"]) * mean).sum()
    return loss.float().reshape(1), counts, mean.float()


def _balance_backward(s):
    e = s["experts"]
    p, c = _probs(s).double(), s["counts"][:e].double()
    kept = s["counts"][e].double()
    some = torch.where(kept > 0, kept, torch.ones_like(kept))
    by = s["dloss"].double() * COEF * e / (some * some * s["slots"])
    c = c - (c.sum() / e).floor()  # p sums to 1: what all counts have in common cancels
    return (by * p * (c - (p * c).sum(1, keepdim=True))).to(s["x"].dtype)


def _grad_clip(s):
    g = torch.cat([t.float() for t in s["g"]])
    norm = g.double().square().sum().sqrt()
    if not s["clip"]:
        return norm.float().reshape(1)
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    s["flat"].copy_(g * scale)
    return norm.float().reshape(1), s["flat"]


PLAIN = {"linear": _linear, "act_backward": _act_backward, "balance": _balance, "balance_backward": _balance_backward,
         "grad_clip": _grad_clip}


def work(case):
    op = case["op"]
    if op == "linear":
        m, rows, cols, r = case["m"], case["rows"], case["cols"], case["rank"]
        n = rows * cols
        per = 0.5 + (1 / 16 if case["scales"] == "plain" else 1 / 64 + 4 / 16384)
        outs = 1 + case["residual"] + case["pre"]
        return {"bytes": n * per + 2.0 * (m * cols + outs * m * rows + r * (rows + cols)) + 4.0 * rows * (case["bias"] != "none"),
                "flops": 2.0 * m * n + 2.0 * m * r * (rows + cols)}
    if op == "act_backward":
        n = case["m"] * case["rows"]
        return {"bytes": 6.0 * n + 4.0 * case["rows"], "flops": 10.0 * n}
    if op in ("balance", "balance_backward"):
        n = case["tokens"] * case["experts"]
        row = (2 if case["logits"] != "f32" else 4) * (1.0 - case["masked"])
        if op == "balance":
            return {"bytes": n * row + 4.0 * case["tokens"] * case["slots"] + 8.0 * case["experts"], "flops": 5.0 * n}
        return {"bytes": n * (row + (2.0 if case["logits"] != "f32" else 4.0)) + 4.0 * case["experts"], "flops": 8.0 * n}
    sizes = _grad_sizes(case)
    types = _grad_types(case, len(sizes))
    size = {torch.float32: 4.0, torch.bfloat16: 2.0, torch.float16: 2.0}
    read = sum(n * size[t] for n, t in zip(sizes, types))
    return {"bytes": read + (sum(sizes) * size[types[0]] if case["clip"] else 4.0), "flops": 3.0 * sum(sizes)}


# ------------------------------------------------------ the results in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        return _exact_linear(case, s)
    if op == "act_backward":
        z, dy = s["z"].double(), s["dy"].double()
        with torch.enable_grad():  # the slope as the derivative of the definition
            z.requires_grad_(True)
            (dz,) = torch.autograd.grad(_exact_act(case["act"], z), z, dy)
        return dz, dz.sum(0)
    if op in ("balance", "balance_backward"):
        return _exact_balance(case, s)
    total = 0.0
    for t in s["g"]:
        total += float(t.double().norm()) ** 2
    norm = torch.tensor([math.sqrt(total)], dtype=torch.float64)
    if not case["clip"]:
        return norm
    scale = min(1.0, s["max_norm"] / (math.sqrt(total) + 1e-6))
    return norm, torch.cat([t.double() * scale for t in s["g"]])


def _exact_act(kind, z):
    if kind == "none":
        return z
    if kind == "relu":
        return z.clamp(min=0)
    if kind == "silu":
        return z * torch.sigmoid(z)
    if kind == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.sigmoid(2 * u)


def _exact_linear(case, s):
    rows, cols = case["rows"], case["cols"]
    byte = s["packed"].long()
    levels = s["levels"].double()
    w = torch.empty(rows * cols, dtype=torch.float64, device=byte.device)
    w[0::2], w[1::2] = levels[byte // 16], levels[byte % 16]
    if "absmax" in s:
        a = s["absmax"].double()
    else:
        code = s["qabsmax"]
        r = code.double() / 127 if case["scales"] == "int8" else s["ratios"][code.long()]
        a = r * s["absmax2"].double()[torch.arange(r.numel(), device=r.device) // 256] + s["mean"].double()
    w = (w.reshape(-1, 64) * a[:, None]).reshape(rows, cols)
    if case["rank"]:  # the adapters merged into the weight
        w += LORA_SCALE * (s["lb"].double() @ s["la"].double())
    z = s["x"].double() @ w.t()
    if s["b"] is not None:
        z += s["b"].double()
    y = _exact_act(case["act"], z)
    if s["r"] is not None:
        y = y + s["r"].double()
    return (y, z) if case["pre"] else y


def _exact_balance(case, s):
    """Token rows by log-sum-exp; the gradient as the derivative of the loss."""
    e, k = case["experts"], case["slots"]
    x = s["x"].double()
    kept = s["mask"] if s["mask"] is not None else torch.ones(x.shape[0], dtype=torch.bool, device=x.device)
    rows = kept & (x > -math.inf).any(1)
    t = int(kept.sum())
    with torch.enable_grad():
        live = x[rows].requires_grad_(True)
        p = torch.exp(live - torch.logsumexp(live, 1, keepdim=True))
        mean = p.sum(0) / max(t, 1)
        ids = s["ids"][kept].reshape(-1)
        c = torch.stack([(ids == i).sum() for i in range(e)]).double()
        loss = COEF * e * (c / max(t * k, 1) * mean).sum()
    if case["op"] == "balance":
        return loss.detach().reshape(1), None, mean.detach()
    out = torch.zeros_like(x)
    if live.shape[0]:
        (grad,) = torch.autograd.grad(loss * s["dloss"].double()[0], live)
        out[rows] = grad
    return out
