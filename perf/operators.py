"""The expert products and the group-scaled int4 weights: cases to time and to
compare, and the operators' plain forms.

Families (a case names its own in "op"):

  int4_gemv           y = x . W^T for 1 <= m <= 16 rows, W[r][c] = (q - z) s with
                      a scale s and a zero point z per `group` columns of a row
  int4_coding         a weight quantized to that form and expanded again
  expert_plan         expert ids of the slots -> order, position, offsets
  expert_gemm         y[p] = x[row(p)] . deq(W_e)^T for the rows p of expert e
  expert_gemm_dx      dx[p] = dy[p] . deq(W_e), its input gradient
  expert_combine      out[t] = sum_j weight[t][j] y[position[t][j]]
  expert_combine_backward   the gradients of that sum

With `own` false, run() computes the plain form in 32 bits; with `own` true it
calls the library."""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _lib():
    """The library, imported where its calls are made."""
    import dequant_matmul_nf4_amd as nf4
    return nf4


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token through an attention projection of an int4 checkpoint: latency
        dict(name="int4_gemv_token", op="int4_gemv", rows=4096, cols=4096, group=128, asym=False, m=1,
             x="bf16", scale="f16", y="bf16"),
        # a decode batch of 16 through a wide gate projection, with zero points
        dict(name="int4_gemv_batch16", op="int4_gemv", rows=28672, cols=8192, group=64, asym=True, m=16,
             x="f16", scale="f16", y="f16"),
        # loading a model: one wide projection quantized, and expanded to measure its error
        dict(name="int4_coding_wide", op="int4_coding", rows=28672, cols=8192, group=128, asym=True, w="bf16", scale="bf16"),
        # one float32 projection, the smallest groups
        dict(name="int4_coding_square", op="int4_coding", rows=4096, cols=4096, group=32, asym=False, w="f32", scale="f16"),
        # routing of one decode batch (latency), and of a long prompt over many experts, some slots dropped
        dict(name="expert_plan_decode", op="expert_plan", slots=64, experts=8, dropped=0.0),
        dict(name="expert_plan_prompt", op="expert_plan", slots=131072, experts=128, dropped=0.05),
        # decode: 8 tokens, two of eight experts each: the weights are read once
        dict(name="expert_gemm_decode", op="expert_gemm", tokens=8, slots=2, experts=8, rows=14336, cols=4096,
             scales="int8", fp4=False, gather=True, skew=0.5),
        # a prompt of 4096 tokens through the same experts: the matrix cores
        dict(name="expert_gemm_prompt", op="expert_gemm", tokens=4096, slots=2, experts=8, rows=14336, cols=4096,
             scales="int8", fp4=False, gather=True, skew=0.5),
        # the backward of that prompt's product
        dict(name="expert_gemm_dx_prompt", op="expert_gemm_dx", tokens=4096, slots=2, experts=8, rows=14336, cols=4096,
             scales="int8", fp4=False, skew=0.5),
        # many small experts, about 64 rows each, unevenly loaded
        dict(name="expert_gemm_dx_fine", op="expert_gemm_dx", tokens=512, slots=8, experts=64, rows=1024, cols=2048,
             scales="plain", fp4=False, skew=1.0),
        # the experts' outputs of a long prompt joined to its tokens, and the gradients of that
        dict(name="expert_combine_prompt", op="expert_combine", tokens=16384, slots=2, cols=4096, dropped=0.0, weights=True),
        dict(name="expert_combine_backward_prompt", op="expert_combine_backward", tokens=16384, slots=2, cols=4096, dropped=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _of(v, n):
    return max(n, v // n * n)


def draw(rng):
    op = rng.choice(["int4_gemv", "int4_gemv", "int4_coding", "expert_plan", "expert_gemm", "expert_gemm", "expert_gemm_dx",
                     "expert_combine", "expert_combine_backward"])
    if op == "int4_gemv":
        group = rng.choice([32, 64, 128])
        return dict(op=op, rows=_log(rng, 1, 28672), cols=_of(_log(rng, group, 28672), group), group=group,
                    asym=rng.random() < 0.5, m=_log(rng, 1, 16), x=rng.choice(["bf16", "f16"]),
                    scale=rng.choice(["f16", "bf16", "f32"]), y=rng.choice(["bf16", "f16", "f32"]))
    if op == "int4_coding":
        group = rng.choice([32, 64, 128])
        return dict(op=op, rows=_log(rng, 1, 28672), cols=_of(_log(rng, group, 8192), group), group=group,
                    asym=rng.random() < 0.5, w=rng.choice(["bf16", "f16", "f32"]), scale=rng.choice(["f16", "bf16", "f32"]))
    if op == "expert_plan":
        return dict(op=op, slots=_log(rng, 1, 131072), experts=_log(rng, 2, 512), dropped=rng.choice([0.0, 0.05, 0.5]))
    if op in ("expert_combine", "expert_combine_backward"):
        slots = rng.randint(1, 8)
        case = dict(op=op, tokens=_log(rng, 1, 32768 // slots), slots=slots, cols=_of(_log(rng, 64, 8192), 8) // 2,
                    dropped=rng.choice([0.0, 0.05, 0.5]))
        case["cols"] = _of(case["cols"], 8)
        if op == "expert_combine":
            case["weights"] = rng.random() < 0.75
        return case
    experts = _log(rng, 1, 128)
    slots = rng.randint(1, min(8, experts))
    cols = _of(_log(rng, 64, 14336), 64)
    rows = _log(rng, 1, 14336)
    rows = min(rows, max(1, 8 * 14336 * 4096 // (experts * cols)))
    if op == "expert_gemm_dx":
        rows = _of(rows, 8)
    case = dict(op=op, tokens=_log(rng, 1, 4096), slots=slots, experts=experts, rows=rows, cols=cols,
                scales=rng.choice(["int8", "fp8", "plain"]), fp4=rng.random() < 0.25, skew=rng.choice([0.0, 0.5, 1.5]))
    case["tokens"] = max(1, min(case["tokens"], int(4096 * 2 * 14336 * 4096 / (slots * rows * cols))))
    if op == "expert_gemm":
        case["gather"] = rng.random() < 0.5
    return case


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
    """Codes and scales of `experts` stacked weights, as the quantizer leaves them."""
    total = case["experts"] * case["rows"] * case["cols"]
    nb = total // 64
    s = dict(packed=torch.randint(0, 256, (total // 2,), generator=g, device=dev, dtype=torch.uint8),
             levels=(_fp4_levels() if case["fp4"] else _nf4_levels()).to(dev))
    absmax = 0.02 * (2.0 + torch.rand(nb, generator=g, device=dev) * 1.5)
    if case["scales"] == "plain":
        s["absmax"] = absmax
        return s
    s["mean"] = absmax.mean().reshape(1)
    s["absmax2"] = 0.01 + 0.01 * torch.rand(-(-nb // 256), generator=g, device=dev)
    if case["scales"] == "int8":
        s["qabsmax"] = torch.randint(-127, 128, (nb,), generator=g, device=dev, dtype=torch.int16).to(torch.int8)
    else:
        q = torch.randint(0, 127, (nb,), generator=g, device=dev, dtype=torch.int16)
        sign = torch.randint(0, 2, (nb,), generator=g, device=dev, dtype=torch.int16) * 128
        s["qabsmax"] = (q + sign).to(torch.uint8)
        s["ratios"] = _e4m3_ratios().to(dev)
    return s


def _route(tokens, slots, experts, skew, g, dev):
    """Each token's `slots` distinct experts; `skew` makes some experts busier."""
    u = torch.rand((tokens, experts), generator=g, device=dev)
    bias = skew * torch.randn((1, experts), generator=g, device=dev)
    return (bias - torch.log(-torch.log(u.clamp(1e-7, 1 - 1e-7)))).topk(slots, dim=1).indices.reshape(-1).to(torch.int32)


def _drop(ids, share, g, dev):
    return torch.where(torch.rand(ids.shape, generator=g, device=dev) < share, torch.full_like(ids, -1), ids)


def _plan(ids, experts):
    """order, position, offsets of the slots' expert ids (see expert_plan)."""
    n = ids.numel()
    kept = (ids >= 0) & (ids < experts)
    key = torch.where(kept, ids.long(), torch.full_like(ids, experts).long())
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts[:experts].cumsum(0)])
    at = torch.arange(n, device=ids.device)
    position = torch.empty_like(order).scatter_(0, order, at)
    position = torch.where(kept, position, torch.full_like(position, -1))
    order = torch.where(at < offsets[-1], order, torch.full_like(order, -1))
    return order.to(torch.int32), position.to(torch.int32), offsets.to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed) * 7919 + 11)
    op = case["op"]
    s = dict(case)

    def normal(shape, dtype, sigma=1.0):
        return (torch.randn(shape, generator=g, device=dev) * sigma).to(dtype)

    if op == "int4_gemv":
        rows, cols = case["rows"], case["cols"]
        s["packed"] = torch.randint(0, 256, (rows * cols // 2,), generator=g, device=dev, dtype=torch.uint8)
        shape = (rows, cols // case["group"])
        s["scales"] = (0.004 + 0.008 * torch.rand(shape, generator=g, device=dev)).to(DTYPES[case["scale"]])
        s["zeros"] = torch.randint(0, 16, shape, generator=g, device=dev, dtype=torch.uint8) if case["asym"] else None
        s["x"] = normal((case["m"], cols), DTYPES[case["x"]])
    elif op == "int4_coding":
        w = torch.randn((case["rows"], case["cols"]), generator=g, device=dev) * 0.02
        out = torch.rand((case["rows"], case["cols"]), generator=g, device=dev) < 0.001
        s["weight"] = torch.where(out, w * 20, w).to(DTYPES[case["w"]])
    elif op == "expert_plan":
        ids = torch.randint(0, case["experts"], (case["slots"],), generator=g, device=dev, dtype=torch.int32)
        s["ids"] = _drop(ids, case["dropped"], g, dev)
    elif op in ("expert_gemm", "expert_gemm_dx"):
        s |= _make_weight(case, g, dev)
        ids = _route(case["tokens"], case["slots"], case["experts"], case["skew"], g, dev)
        s["order"], _, s["offsets"] = _plan(ids, case["experts"])
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        m = ids.numel()
        if op == "expert_gemm":
            s["x"] = normal((case["tokens"] if case["gather"] else m, case["cols"]), torch.bfloat16)
        else:
            s["dy"] = normal((m, case["rows"]), torch.bfloat16)
    else:
        n = case["tokens"] * case["slots"]
        ids = torch.randint(0, 64, (n,), generator=g, device=dev, dtype=torch.int32)
        _, s["position"], _ = _plan(_drop(ids, case["dropped"], g, dev), 64)
        s["y"] = normal((n, case["cols"]), torch.bfloat16)
        s["gate"] = torch.softmax(torch.randn((case["tokens"], case["slots"]), generator=g, device=dev), 1)
        if op == "expert_combine":
            s["gate"] = s["gate"] if case["weights"] else None
        else:
            s["dout"] = normal((case["tokens"], case["cols"]), torch.bfloat16)
            s["dy"] = torch.zeros((n, case["cols"]), dtype=torch.bfloat16, device=dev)  # rows of dropped slots stay as they are
    return s


# ----------------------------------------------------------- the operators

def run(s):
    if own:
        return _run_own(s)
    return PLAIN[s["op"]](s)


def _run_own(s):
    lib = _lib()
    op = s["op"]
    if op == "int4_gemv":
        w = lib.Int4Weight(s["packed"], s["rows"], s["cols"], s["group"], s["scales"], s["zeros"])
        return lib.nf4_int4_gemv(w, s["x"], y_dtype=DTYPES[s["y"]])
    if op == "int4_coding":
        w = lib.quantize_int4(s["weight"], group=s["group"], symmetric=not s["asym"], scale_dtype=DTYPES[s["scale"]])
        out = {"values": lib.nf4_int4_dequantize(w, out_dtype=torch.float32), "scales": w.scales}
        return out | {"zeros": w.zeros} if s["asym"] else out
    if op == "expert_plan":
        return lib.nf4_expert_plan(s["ids"], s["experts"])
    if op == "expert_combine":
        return lib.nf4_expert_combine(s["y"], s["position"], s["slots"], weights=s["gate"])
    if op == "expert_combine_backward":
        return lib.nf4_expert_combine_backward(s["dout"], s["y"], s["position"], s["slots"], s["gate"], dy=s["dy"])
    w = lib.NF4Weight(s["packed"], s["experts"] * s["rows"], s["cols"], absmax=s.get("absmax"), qabsmax=s.get("qabsmax"),
                      absmax2=s.get("absmax2"), mean=s.get("mean"), dq_type=int(s["scales"] == "fp8"), quant_type=int(s["fp4"]))
    if op == "expert_gemm_dx":
        return lib.nf4_expert_gemm_dx(w, s["experts"], s["dy"], s["offsets"])
    if s["gather"]:
        return lib.nf4_expert_gemm(w, s["experts"], s["x"], s["offsets"], index=s["order"], slots=s["slots"])
    return lib.nf4_expert_gemm(w, s["experts"], s["x"], s["offsets"])


def _unpack(packed):
    """Element 2j is the high half of byte j, element 2j + 1 the low half."""
    return torch.stack((packed >> 4, packed & 15), dim=-1).reshape(-1)


def _int4_gemv(s):
    q = _unpack(s["packed"]).reshape(s["rows"], -1, s["group"]).float()
    z = s["zeros"].float()[..., None] if s["zeros"] is not None else 8.0
    w = ((q - z) * s["scales"].float()[..., None]).reshape(s["rows"], s["cols"])
    return torch.matmul(s["x"].float(), w.t()).to(DTYPES[s["y"]])


def _int4_coding(s):
    x = s["weight"].float().reshape(s["rows"], -1, s["group"])
    kind = DTYPES[s["scale"]]
    if s["asym"]:
        low, high = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
        # (a division by a tensor: one by a Python number is a product with its reciprocal on the GPU)
        scales = ((high - low) / torch.full_like(low, 15)).to(kind)
    else:
        top = x.abs().amax(-1)
        scales = (top / torch.full_like(top, 7)).to(kind)
    by = scales.float()
    some = by > 0
    by = torch.where(some, by, torch.ones_like(by))
    if s["asym"]:
        z = torch.where(some, torch.round(-low / by).clamp(0, 15), torch.zeros_like(by))
    else:
        z = torch.full_like(by, 8)
    q = (torch.round(x / by[..., None]) + z[..., None]).clamp(0, 15)
    q = torch.where(some[..., None], q, z[..., None])
    out = {"values": ((q - z[..., None]) * scales.float()[..., None]).reshape(s["rows"], s["cols"]), "scales": scales}
    return out | {"zeros": z.to(torch.uint8)} if s["asym"] else out


def _expert_plan(s):
    return _plan(s["ids"], s["experts"])


def _dequantized(s):
    """The stacked weights [experts][rows][cols] in float32."""
    if "absmax" in s:
        a = s["absmax"]
    else:
        r = s["qabsmax"].float() / 127 if s["qabsmax"].dtype == torch.int8 else s["ratios"].float()[s["qabsmax"].long()]
        a = r * s["absmax2"].repeat_interleave(256)[:r.numel()] + s["mean"]
    v = s["levels"][_unpack(s["packed"]).to(torch.int32)].reshape(-1, 64)
    return (v * a[:, None]).reshape(s["experts"], s["rows"], s["cols"])


def _by_expert(s):
    """Sorted row and expert of each place of an [experts][most] table, and where it holds a row."""
    first = s["offsets"][:-1].long()[:, None]
    p = first + torch.arange(s["most"], device=first.device)[None, :]
    return p, p < s["offsets"][1:].long()[:, None]


def _padded(rows, p, live):
    t = rows.float()[p.clamp(max=rows.shape[0] - 1)]
    return torch.where(live[..., None], t, torch.zeros_like(t))


def _expert_gemm(s):
    p, live = _by_expert(s)
    x = s["x"][(s["order"].long() // s["slots"])] if s["gather"] else s["x"]
    xt = _padded(x, p, live).transpose(1, 2).contiguous()
    y = torch.bmm(_dequantized(s), xt).transpose(1, 2)
    return torch.zeros((x.shape[0], s["rows"]), device=x.device).index_put_((p[live],), y[live]).to(torch.bfloat16)


def _expert_gemm_dx(s):
    p, live = _by_expert(s)
    dx = torch.bmm(_padded(s["dy"], p, live), _dequantized(s))
    return torch.zeros((s["dy"].shape[0], s["cols"]), device=dx.device).index_put_((p[live],), dx[live]).to(torch.bfloat16)


def _picked(s):
    """The slots' rows of y in float32 [tokens][slots][cols], dropped ones as zeros."""
    at = s["position"].long().reshape(s["tokens"], s["slots"])
    rows = s["y"].float()[at.clamp(min=0)]
    return torch.where((at >= 0)[..., None], rows, torch.zeros_like(rows)), at


def _expert_combine(s):
    rows, _ = _picked(s)
    if s["gate"] is not None:
        rows = rows * s["gate"][..., None]
    return rows.sum(1).to(torch.bfloat16)


def _expert_combine_backward(s):
    rows, at = _picked(s)
    dout = s["dout"].float()
    live = at.reshape(-1) >= 0
    grad = (s["gate"][..., None] * dout[:, None, :]).reshape(-1, s["cols"]).to(torch.bfloat16)
    s["dy"][at.reshape(-1)[live]] = grad[live]
    return s["dy"], (rows * dout[:, None, :]).sum(-1)


PLAIN = {"int4_gemv": _int4_gemv, "int4_coding": _int4_coding, "expert_plan": _expert_plan, "expert_gemm": _expert_gemm,
         "expert_gemm_dx": _expert_gemm_dx, "expert_combine": _expert_combine,
         "expert_combine_backward": _expert_combine_backward}


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if op == "int4_gemv":
        n = case["rows"] * case["cols"]
        per = size[case["scale"]] + (1 if case["asym"] else 0)
        return {"bytes": n / 2 + n / case["group"] * per + case["m"] * (case["cols"] * size[case["x"]] + case["rows"] * size[case["y"]]),
                "flops": 2.0 * case["m"] * n}
    if op == "int4_coding":
        # the weight read once, codes and scales written, read again, the values written
        n = case["rows"] * case["cols"]
        per = size[case["scale"]] + (1 if case["asym"] else 0)
        return {"bytes": n * size[case["w"]] + 2 * (n / 2 + n / case["group"] * per) + 4.0 * n, "flops": 6.0 * n}
    if op == "expert_plan":
        return {"bytes": 12.0 * case["slots"] + 4.0 * (case["experts"] + 1), "flops": 0.0}
    if op in ("expert_combine", "expert_combine_backward"):
        n, kept = case["tokens"] * case["slots"], 1 - case["dropped"]
        row = 2.0 * case["cols"]
        both = 2 if op == "expert_combine_backward" else 1
        return {"bytes": both * kept * n * row + case["tokens"] * row + n * 4.0 * (1 + both), "flops": 2.0 * both * n * case["cols"]}
    m = case["tokens"] * case["slots"]
    touched = case["experts"] * (1 - (1 - case["slots"] / case["experts"]) ** case["tokens"])
    n = case["rows"] * case["cols"]
    per = 0.5 + (1 / 16 if case["scales"] == "plain" else 1 / 64 + 4 / 16384)
    read = case["tokens"] if op == "expert_gemm" and case["gather"] else m
    ins, outs = (case["cols"], case["rows"]) if op == "expert_gemm" else (case["rows"], case["cols"])
    return {"bytes": touched * n * per + 2.0 * (read * ins + m * outs), "flops": 2.0 * m * n}


# ------------------------------------------------------ the results in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "expert_plan":
        return None
    if op == "int4_gemv":
        codes = torch.empty(case["rows"], case["cols"], dtype=torch.float64, device=s["x"].device)
        b = s["packed"].reshape(case["rows"], -1)
        codes[:, 0::2], codes[:, 1::2] = (b // 16).double(), (b % 16).double()
        spread = lambda t: t.double().repeat_interleave(case["group"], dim=1)  # noqa: E731
        codes -= spread(s["zeros"]) if case["asym"] else 8
        codes *= spread(s["scales"])
        return s["x"].double() @ codes.t()
    if op == "int4_coding":
        return _exact_coding(case, s)
    if op in ("expert_gemm", "expert_gemm_dx"):
        return _exact_product(case, s)
    at = s["position"].reshape(case["tokens"], case["slots"]).long()
    y = torch.cat([s["y"].double(), torch.zeros(1, case["cols"], dtype=torch.float64, device=s["y"].device)])  # row -1: dropped
    if op == "expert_combine":
        out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device=y.device)
        for j in range(case["slots"]):
            out += y[at[:, j]] * (s["gate"][:, j:j + 1].double() if s["gate"] is not None else 1.0)
        return out
    dout = s["dout"].double()
    dy = torch.zeros_like(y)
    dgate = []
    for j in range(case["slots"]):
        dy[at[:, j]] = dout * s["gate"][:, j:j + 1].double()
        dgate.append((dout * y[at[:, j]]).sum(1))
    return dy[:-1], torch.stack(dgate, 1)


def _exact_coding(case, s):
    """Group by group along the rows, the scale rounded to its type."""
    x = s["weight"].double()
    parts = x.split(case["group"], dim=1)
    values, scales, zeros = [], [], []
    for p in parts:
        if case["asym"]:
            low = torch.minimum(p.min(1).values, torch.zeros_like(p[:, 0]))
            high = torch.maximum(p.max(1).values, torch.zeros_like(p[:, 0]))
            a = ((high - low) / 15).to(DTYPES[case["scale"]]).double()
            z = torch.nan_to_num((-low / a)).round().clamp(0, 15)
        else:
            a = (p.abs().max(1).values / 7).to(DTYPES[case["scale"]]).double()
            z = torch.full_like(a, 8.0)
        q = (torch.nan_to_num(p / a[:, None]).round() + z[:, None]).clamp(0, 15)
        values.append((q - z[:, None]) * a[:, None])
        scales.append(a)
        zeros.append(z.to(torch.uint8))
    out = {"values": torch.cat(values, 1), "scales": torch.stack(scales, 1)}
    return out | {"zeros": None} if case["asym"] else out


def _exact_product(case, s):
    """Expert by expert."""
    bounds = s["offsets"].tolist()
    rows, cols = case["rows"], case["cols"]
    src = s["x"] if case["op"] == "expert_gemm" else s["dy"]
    out = torch.zeros(bounds[-1], rows if case["op"] == "expert_gemm" else cols, dtype=torch.float64, device=src.device)
    levels = s["levels"].double()
    for e in range(case["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        byte = s["packed"][e * rows * cols // 2:(e + 1) * rows * cols // 2].long()
        w = torch.empty(rows * cols, dtype=torch.float64, device=src.device)
        w[0::2], w[1::2] = levels[byte // 16], levels[byte % 16]
        b0, b1 = e * rows * cols // 64, (e + 1) * rows * cols // 64
        if "absmax" in s:
            a = s["absmax"][b0:b1].double()
        else:
            code = s["qabsmax"][b0:b1]
            r = code.double() / 127 if case["scales"] == "int8" else s["ratios"][code.long()]
            a = r * s["absmax2"].double()[torch.arange(b0, b1, device=src.device) // 256] + s["mean"].double()
        w = (w.reshape(-1, 64) * a[:, None]).reshape(rows, cols)
        if case["op"] == "expert_gemm":
            at = s["order"][lo:hi].long() // case["slots"] if case["gather"] else torch.arange(lo, hi, device=src.device)
            out[lo:hi] = src[at].double() @ w.t()
        else:
            out[lo:hi] = src[lo:hi].double() @ w
    return out
