"""nf4_expert_balance and its gradient against float64.

Bounds: a probability's relative error is that of two exponentials (arguments of
size v: (1.45 v + 2) 2^-24 each), a sum of E terms and a division; the sums over
tokens in float32 stay below (tokens of a lane + 32) 2^-24.  Counts are exact."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.layer_common import F32, HALF, types, worst

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(41)


def make(torch, tokens, experts, slots, kind, masked=0.0, dropped=0.0, closed=0.0, sigma=2.0):
    x = (sigma * torch.randn((tokens, experts), device="cuda")).to(types(torch)[kind])
    if closed:
        x = torch.where(torch.rand(x.shape, device="cuda") < closed, torch.full_like(x, -INF), x)
        x[torch.rand(tokens, device="cuda") < 0.05] = -INF
    ids = torch.randint(0, experts, (tokens, slots), dtype=torch.int32, device="cuda")
    ids = torch.where(torch.rand(ids.shape, device="cuda") < dropped, torch.full_like(ids, experts + 3), ids)
    ids = torch.where(torch.rand(ids.shape, device="cuda") < dropped, torch.full_like(ids, -1), ids)
    mask = torch.rand(tokens, device="cuda") >= masked if masked else None
    return x, ids, mask


def reference(torch, x, ids, slots, coef, mask, dloss=1.0):
    tokens, experts = x.shape
    kept = mask.bool() if mask is not None else torch.ones(tokens, dtype=torch.bool, device=x.device)
    z = x.double()
    live = kept & (z > -INF).any(1)
    p = torch.zeros_like(z)
    p[live] = torch.softmax(z[live], 1)
    t = int(kept.sum())
    flat = ids.reshape(tokens, slots)[kept].reshape(-1).long()
    flat = flat[(flat >= 0) & (flat < experts)]
    c = torch.bincount(flat, minlength=experts)
    n = max(t, 1)
    mean = p.sum(0) / n
    loss = coef * experts * (c.double() / (n * slots) * mean).sum()
    grad = dloss * coef * experts / (n * n * slots) * p * (c.double() - (p * c.double()).sum(1, keepdim=True))
    counts = torch.cat([c, torch.tensor([t], device=x.device)]).to(torch.int32)
    return loss, counts, mean, p, grad


def eta(x):
    """Relative error of a probability."""
    z = x.double()
    top = z.masked_fill(z == -INF, 0.0).abs().max()
    return (4 * (1.45 * 2 * float(top) + 3) + 2 * x.shape[1]) * F32


def check(torch, x, ids, slots, coef, mask, dloss=None):
    kind = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}[x.dtype]
    loss, counts, mean = nf4.nf4_expert_balance(x, ids, slots, coef, mask=mask)
    by = 1.0 if dloss is None else float(dloss)
    rl, rc, rm, p, rg = reference(torch, x, ids, slots, coef, mask, by)
    assert torch.equal(counts, rc)
    e = eta(x) + (x.shape[0] / 64 + 64) * F32
    assert worst((mean.double() - rm).abs(), e * rm + 1e-30) <= 1.0
    assert worst((loss.double() - rl).abs(), (e + 4 * F32) * rl.abs().reshape(1) + 1e-30) <= 1.0
    g = nf4.nf4_expert_balance_backward(x, counts, slots, coef, mask=mask, dloss=dloss)
    assert g.dtype == x.dtype
    c = rc[:-1].double()
    c = (c - torch.floor(c.mean())).abs()
    t = max(1, int(rc[-1]))
    factor = abs(by * coef) * x.shape[1] / (t * t * slots)
    off = eta(x) * factor * p * (c + (p * c).sum(1, keepdim=True)) + 4 * F32 * rg.abs() + 1e-37
    # the reference's own rounding: E + 4 operations in float64 on values up to the largest count
    off = off + factor * p * float(rc[:-1].max()) * (x.shape[1] + 4) * 2.0 ** -53
    step = {"f32": 0.0, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}[kind]  # half the smallest number's step
    if kind != "f32":
        off = off + HALF[kind] * (rg.abs() + off) + step
    assert worst((g.double() - rg).abs(), off) <= 1.0
    if mask is not None:
        assert (g[~mask.bool()] == 0).all()
    return g


CASES = [(1, 1, 1), (1, 8, 2), (2, 2, 1), (7, 3, 2), (64, 8, 2), (100, 5, 1), (333, 16, 4), (1000, 60, 6), (4096, 64, 8), (50, 127, 3),
         (3000, 128, 8), (200, 129, 2), (777, 256, 8), (130, 300, 4), (90, 511, 8), (70, 512, 2), (33, 1000, 1), (300, 1024, 8), (20000, 8, 2),
         (70001, 2, 1)]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("tokens,experts,slots", CASES)
def test_against_float64(kind, tokens, experts, slots):
    torch = need_gpu()
    say("balance", kind, tokens, experts, slots)
    x, ids, mask = make(torch, tokens, experts, slots, kind)
    # a gradient of the loss that keeps fp16's in range
    check(torch, x, ids, slots, 0.01, mask, torch.full((1,), 50.0 * tokens, device="cuda"))
    x, ids, mask = make(torch, tokens, experts, slots, kind, masked=0.4, dropped=0.1, closed=0.2 if experts > 1 else 0.0)
    check(torch, x, ids, slots, 1.5, mask, torch.full((1,), float(tokens), device="cuda"))


def test_gradient_is_that_of_the_loss():
    """Against differences of the 64-bit loss with the counts held, and against autograd."""
    torch = need_gpu()
    x, ids, mask = make(torch, 12, 6, 2, "f32", masked=0.2)
    coef = 0.7
    _, counts, _ = nf4.nf4_expert_balance(x, ids, 2, coef, mask=mask)
    g = nf4.nf4_expert_balance_backward(x, counts, 2, coef, mask=mask)
    kept, c = mask.double(), counts[:-1].double()

    def loss(z):
        return coef * 6 * (c / (counts[-1] * 2) * (torch.softmax(z, 1) * kept[:, None]).sum(0) / counts[-1]).sum()

    z = x.double().requires_grad_(True)
    (auto,) = torch.autograd.grad(loss(z), z)
    assert worst((g.double() - auto).abs(), 1e-5 * auto.abs() + 1e-7 * float(auto.abs().max())) <= 1.0
    h = 1e-5
    for t, e in ((0, 0), (3, 5), (11, 2)):
        d = torch.zeros_like(x, dtype=torch.float64)
        d[t, e] = h
        num = (loss(x.double() + d) - loss(x.double() - d)) / (2 * h)
        assert abs(float(g[t, e]) - float(num)) <= 1e-5 * abs(float(num)) + 1e-8


@pytest.mark.parametrize("tokens,experts", [(5, 8), (3000, 40)])
def test_nothing_kept(tokens, experts):
    torch = need_gpu()
    x, ids, _ = make(torch, tokens, experts, 2, "f32")
    x[0] = float("nan")
    mask = torch.zeros(tokens, dtype=torch.uint8, device="cuda")
    loss, counts, mean = nf4.nf4_expert_balance(x, ids, 2, 0.01, mask=mask)
    assert float(loss) == 0 and (counts == 0).all() and (mean == 0).all()
    g = nf4.nf4_expert_balance_backward(x, counts, 2, 0.01, mask=mask)
    assert (g == 0).all()
    # rows without any probability count as tokens, and have no gradient
    x = torch.full((tokens, experts), -INF, device="cuda")
    loss, counts, mean = nf4.nf4_expert_balance(x, ids, 2, 0.01)
    assert float(loss) == 0 and int(counts[-1]) == tokens and (mean == 0).all()
    assert (nf4.nf4_expert_balance_backward(x, counts, 2, 0.01) == 0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_tokens_left_out_may_hold_anything(kind):
    torch = need_gpu()
    for tokens, experts in ((40, 8), (9000, 24)):
        x, ids, mask = make(torch, tokens, experts, 2, kind, masked=0.5)
        first = nf4.nf4_expert_balance(x, ids, 2, 0.01, mask=mask)
        g = nf4.nf4_expert_balance_backward(x, first[1], 2, 0.01, mask=mask)
        junk = x.clone()
        junk[~mask] = float("nan")
        junk[~mask, 0] = INF
        again = nf4.nf4_expert_balance(junk, ids, 2, 0.01, mask=mask)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
        assert torch.equal(g, nf4.nf4_expert_balance_backward(junk, first[1], 2, 0.01, mask=mask))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("experts", [7, 9, 64, 100])
def test_logits_at_any_alignment(kind, experts):
    """A view that begins at an odd element."""
    torch = need_gpu()
    x, ids, _ = make(torch, 600, experts, 2, kind)
    room = torch.zeros(x.numel() + 3, dtype=x.dtype, device="cuda")
    view = room[1:1 + x.numel()].view(600, experts)
    view.copy_(x)
    a, b = nf4.nf4_expert_balance(x, ids, 2, 0.1), nf4.nf4_expert_balance(view, ids, 2, 0.1)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    g = nf4.nf4_expert_balance_backward(x, a[1], 2, 0.1)
    out = torch.full_like(room, 7)
    nf4.nf4_expert_balance_backward(view, a[1], 2, 0.1, dlogits=out[1:1 + x.numel()].view(600, experts))
    assert torch.equal(out[1:1 + x.numel()].view(600, experts), g) and out[0] == 7 and (out[1 + x.numel():] == 7).all()
    nf4.nf4_expert_balance_backward(view, a[1], 2, 0.1, dlogits=view)  # in place
    assert torch.equal(view, g)


def test_equal_counts_and_one_expert():
    """Where all counts are equal the gradient is zero, as the definition has it."""
    torch = need_gpu()
    x = torch.randn((4096, 32), device="cuda")
    ids = (torch.arange(4096 * 4, device="cuda", dtype=torch.int32) % 32).reshape(4096, 4).contiguous()
    loss, counts, mean = nf4.nf4_expert_balance(x, ids, 4, 1.0)
    assert (counts[:-1] == 512).all()
    assert (nf4.nf4_expert_balance_backward(x, counts, 4, 1.0) == 0).all()


def test_no_tokens():
    torch = need_gpu()
    x = torch.empty((0, 8), device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    loss, counts, mean = nf4.nf4_expert_balance(x, ids, 2, 0.01)
    assert float(loss) == 0 and tuple(counts.shape) == (9,) and (counts == 0).all() and (mean == 0).all()
    assert tuple(nf4.nf4_expert_balance_backward(x, counts, 2, 0.01).shape) == (0, 8)
