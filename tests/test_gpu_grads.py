"""nf4_grad_norm and nf4_grad_clip against float64.

Bounds: squares and their sum are float64, the norm is rounded once to float32;
a scaled gradient has the scale's rounding (2^-24), the product's (2^-24) and
its type's (the smallest numbers of a type: half their step)."""

from __future__ import annotations

import math

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.layer_common import F32, HALF, types, worst

pytestmark = pytest.mark.gpu
TINY = {"f32": 2.0 ** -150, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(43)


def make(torch, sizes, kinds):
    return [(torch.randn(n, device="cuda") * (0.1 + 0.2 * (i % 7))).to(types(torch)[kinds[i % len(kinds)]]) for i, n in enumerate(sizes)]


def norm64(grads):
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def near(got, want):
    assert abs(float(got) - want) <= (F32 + 1e-12) * want + 2.0 ** -150, (float(got), want)


def check_scaled(torch, outs, grads, norm, most):
    scale = min(1.0, most / (norm + 1e-6))
    for o, g in zip(outs, grads):
        kind = {torch.bfloat16: "bf16", torch.float16: "f16", torch.float32: "f32"}[o.dtype]
        ref = g.double().reshape(-1) * scale
        off = 2.5 * F32 * ref.abs()
        off = off + (HALF[kind] * (ref.abs() + off) if kind != "f32" else 0.0) + TINY[kind]
        assert worst((o.double().reshape(-1) - ref).abs(), off) <= 1.0, (kind, g.numel())


SETS = {
    "one value": ([1], ["f32"]), "one of each": ([5, 6, 7], ["f32", "bf16", "f16"]),
    "odd": ([1, 3, 2047, 2048, 2049, 16383, 16384, 16385, 100003], ["bf16", "f32"]),
    "large": ([5_000_001, 3, 2_000_000], ["f32"]), "half": ([70000, 1, 40], ["f16"]),
    "with empty ones": ([0, 10, 0, 0, 33000, 0], ["f32", "f16"]), "all empty": ([0, 0], ["f32"]),
    "as many as arguments hold": ([100 + i for i in range(112)], ["f32", "bf16", "f16"]),
    "one more": ([100 + i for i in range(113)], ["bf16", "f32"]),
    "many": ([(i * 7919) % 30011 for i in range(1000)], ["f32", "bf16", "f16", "f32"]),
}


@pytest.mark.parametrize("name", SETS)
def test_against_float64(name):
    torch = need_gpu()
    say("grads", name)
    sizes, kinds = SETS[name]
    grads = make(torch, sizes, kinds)
    n = norm64(grads)
    near(nf4.nf4_grad_norm(grads), n)
    total = sum(sizes)
    for most in (0.37 * n, 2.0 * n + 1, 0.0):
        for kind in ("f32", "bf16", "f16"):
            out = torch.full((total + 3,), 7.0, dtype=types(torch)[kind], device="cuda")
            place = out[:total]
            got, same = nf4.nf4_grad_clip(grads, most, out=place)
            near(got, n)
            assert same is place and (out[total:] == 7).all()
            check_scaled(torch, out[:total].split(sizes), grads, n, most)
        mine = [g.clone() for g in grads]
        near(nf4.nf4_grad_clip(mine, most), n)
        check_scaled(torch, mine, grads, n, most)
        if most > n:
            assert all(torch.equal(a, b) for a, b in zip(mine, grads))


def test_same_twice():
    torch = need_gpu()
    grads = make(torch, [30_011 + 17 * i for i in range(300)], ["f32", "bf16"])
    a, b = nf4.nf4_grad_norm(grads), nf4.nf4_grad_norm(grads)
    assert torch.equal(a, b)
    out = torch.empty(sum(g.numel() for g in grads), device="cuda")
    c, _ = nf4.nf4_grad_clip(grads, 1.0, out=out)
    assert torch.equal(a, c)
    first = out.clone()
    nf4.nf4_grad_clip(grads, 1.0, out=out)
    assert torch.equal(first, out)


def test_squares_past_float32():
    """Gradients whose squares leave float32's range at either end."""
    torch = need_gpu()
    for v in (1e30, 3e38, 1e-30, 1e-42):
        g = torch.full((1000,), v, device="cuda")
        n = norm64([g])
        got = nf4.nf4_grad_norm([g])
        if n < 3.4e38:
            near(got, n)
        else:
            assert float(got) == math.inf
        mine = g.clone()
        nf4.nf4_grad_clip([mine], 1e-20)
        check_scaled(torch, [mine], [g], n, 1e-20)


def test_not_finite():
    torch = need_gpu()
    g = torch.randn(5000, device="cuda")
    inf, nan = g.clone(), g.clone()
    inf[77], nan[4999] = math.inf, math.nan
    mine = inf.clone()
    assert float(nf4.nf4_grad_clip([mine], 1.0)) == math.inf
    assert mine[77].isnan() and (mine[:77] == 0).all() and (mine[78:] == 0).all()
    mine = nan.clone()
    assert math.isnan(float(nf4.nf4_grad_clip([mine], 1e9))) and mine.isnan().all()


def test_given_norm():
    """The norm over more gradients than these: shards of one set are scaled alike."""
    torch = need_gpu()
    grads = make(torch, [4000, 17, 70001], ["f32", "bf16"])
    n = norm64(grads)
    total = torch.full((1,), 10 * n, device="cuda")
    mine = [g.clone() for g in grads]
    got = nf4.nf4_grad_clip(mine, 2 * n, total_norm=total)
    assert torch.equal(got, total)
    check_scaled(torch, mine, grads, float(total), 2 * n)
    again = [g.clone() for g in grads]
    assert nf4.nf4_grad_clip(again, 2 * n, total_norm=total, norm=total) is total
    assert all(torch.equal(a, b) for a, b in zip(mine, again))


def test_views_at_any_alignment():
    torch = need_gpu()
    for kind in ("f32", "bf16", "f16"):
        room = (torch.randn(60000, device="cuda")).to(types(torch)[kind])
        views = [room[1:20000], room[20001:20002], room[20003:50000], room[50005:]]
        want = [v.clone() for v in views]
        n = norm64(want)
        gaps = room[[0, 20000, 20002, 50000, 50004]].clone()
        near(nf4.nf4_grad_clip(views, 0.5 * n), n)
        check_scaled(torch, views, want, n, 0.5 * n)
        assert torch.equal(room[[0, 20000, 20002, 50000, 50004]], gaps)


def test_shapes_and_refusals():
    torch = need_gpu()
    g = torch.randn((30, 40), device="cuda")
    near(nf4.nf4_grad_norm([g, g[:0], g.reshape(2, 3, 200)]), math.sqrt(2) * norm64([g]))
    with pytest.raises(ValueError):
        nf4.nf4_grad_clip([g, g], 1.0)                       # scaled twice
    with pytest.raises(ValueError):
        nf4.nf4_grad_clip([g, g[3:5]], 1.0)
    with pytest.raises(ValueError):
        nf4.nf4_grad_norm([g.t()])
    with pytest.raises(ValueError):
        nf4.nf4_grad_norm([])
    with pytest.raises(ValueError):
        nf4.nf4_grad_clip([g], 1.0, out=torch.empty(5, device="cuda"))
    with pytest.raises(ValueError):
        nf4.nf4_grad_clip([g[1:]], 1.0, out=g.reshape(-1)[:-40])   # over its own source, but not in place
    with pytest.raises(nf4.NF4Error):
        nf4.nf4_grad_clip([g], math.nan)
    with pytest.raises(TypeError):
        nf4.nf4_grad_norm([g.double()])
    both = g.clone()
    nf4.nf4_grad_clip([both[:15], both[15:]], 0.1, out=both.reshape(-1))   # exactly in place
    mine = [g[:15].clone(), g[15:].clone()]
    nf4.nf4_grad_clip(mine, 0.1)
    assert torch.equal(both, torch.cat(mine))


def test_offsets_past_32_bits():
    torch = need_gpu()
    n = (1 << 31) + (1 << 20) + 5
    say("grads", n)
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-1], g[0], g[1 << 31] = 3.0, 4.0, 12.0
    near(nf4.nf4_grad_clip([g], 6.5), 13.0)
    assert float(g[-1]) == 1.5 and float(g[0]) == 2.0 and float(g[1 << 31]) == 6.0
