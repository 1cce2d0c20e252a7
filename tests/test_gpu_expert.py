"""The expert products, their plan and their join on the GPU.

The plan is compared for equality.  The products are compared with a float64
product of the dequantized weights.  Tolerances per output, with
S = sum |x| |w|: half a step of bfloat16 on the value (2^-8), the float32 sum
of K products (K 2^-24 of S), and the rounding of the operands: a weight
rounded once to bfloat16 is off by at most 2^-8 of its value, levels carried as
two bfloat16 parts by at most 2^-16."""

from __future__ import annotations

import numpy as np
import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(20)


def _plan_np(ids, experts):
    ids = np.asarray(ids, np.int64)
    kept = (ids >= 0) & (ids < experts)
    key = np.where(kept, ids, experts)
    order = np.argsort(key, kind="stable")
    position = np.empty_like(order)
    position[order] = np.arange(len(ids))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])])
    order = np.where(np.arange(len(ids)) < offsets[-1], order, -1)
    return order, np.where(kept, position, -1), offsets


@pytest.mark.parametrize("n,experts", [(1, 1), (1, 1024), (7, 2), (64, 8), (1000, 3), (1024, 64), (1025, 65), (4096, 256),
                                       (4097, 256), (20000, 1), (70001, 1024), (300000, 7), (600000, 128)])
@pytest.mark.parametrize("kind", ["even", "dropped", "one"])
def test_plan(n, experts, kind):
    torch = need_gpu()
    say("plan", n, experts, kind)
    g = np.random.default_rng(n + experts)
    ids = g.integers(0, experts, n)
    if kind == "dropped":
        ids = np.where(g.random(n) < 0.3, g.choice([-1, experts, -2 ** 31, 2 ** 31 - 1], n), ids)
    elif kind == "one":
        ids[:] = experts - 1
    got = nf4.nf4_expert_plan(torch.from_numpy(ids.astype(np.int32)).cuda(), experts)
    for a, b, name in zip(got, _plan_np(ids, experts), ("order", "position", "offsets")):
        assert np.array_equal(a.cpu().numpy(), b), name


def test_plan_of_dropped_slots_alone():
    torch = need_gpu()
    for n in (5, 9000):
        order, position, offsets = nf4.nf4_expert_plan(torch.full((n,), -1, dtype=torch.int32, device="cuda"), 6)
        assert (order == -1).all() and (position == -1).all() and (offsets == 0).all()


# ------------------------------------------------------------------ products

def _stack(torch, experts, rows, cols, scales="int8", fp4=False, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn((experts * rows, cols), generator=g, device="cuda") * 0.02).bfloat16()
    return nf4.quantize_weight(w, double_quant=scales != "plain", dq_type=scales if scales != "plain" else "int8",
                               quant_type="fp4" if fp4 else "nf4")


def _counts(kind, experts, m, seed=3):
    g = np.random.default_rng(seed)
    if kind == "even":
        c = np.full(experts, m // experts)
        c[:m % experts] += 1
    elif kind == "one":
        c = np.zeros(experts, int)
        c[experts // 2] = m
    else:  # uneven, some empty
        p = g.random(experts) ** 4 * (g.random(experts) < 0.7)
        p = p / p.sum() if p.sum() else np.full(experts, 1 / experts)
        c = g.multinomial(m, p)
    return np.concatenate([[0], np.cumsum(c)])


def _reference(torch, W, experts, x, offsets, dx=False):
    """float64 product and the sums of magnitudes, row by sorted row."""
    w = nf4.nf4_dequantize(W, out_dtype=torch.float32).double().view(experts, -1, W.cols)
    ref, mag = [], []
    for e in range(experts):
        xe = x[offsets[e]:offsets[e + 1]].double()
        we = w[e] if dx else w[e].t()
        ref.append(xe @ we)
        mag.append(xe.abs() @ we.abs())
    return torch.cat(ref), torch.cat(mag)


def _check(got, ref, mag, terms, w_rel=2.0 ** -8):
    bound = 2.0 ** -8 * ref.abs() + (terms * 2.0 ** -24 + w_rel) * mag + 1e-30
    worst = ((got.double() - ref).abs() / bound).max().item()
    assert worst <= 1.0, worst
    # the roundings are independent: in the whole they stay near one rounding's size, which the bound
    # above (all of them adding up) would not show: output and weight, each at most 2^-8 / sqrt(3) in the mean square
    if ref.numel() >= 1000:
        rel = ((got.double() - ref).norm() / ref.norm()).item()
        assert rel <= (2 / 3) ** 0.5 * 2.0 ** -8 * 1.1, rel


SHAPES = [  # experts, rows, cols, m
    (1, 1, 64, 1), (1, 256, 512, 40), (2, 17, 128, 3), (4, 250, 192, 100), (8, 512, 1024, 16), (8, 64, 4160, 9),
    (3, 300, 640, 1000), (70, 40, 128, 333), (300, 8, 64, 700), (5, 1032, 320, 61), (2, 48, 14336, 37),
]


@pytest.mark.parametrize("experts,rows,cols,m", SHAPES)
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_expert_gemm(experts, rows, cols, m, kind):
    torch = need_gpu()
    say("expert gemm", experts, rows, cols, m, kind)
    scales = ["int8", "fp8", "plain"][(rows + m) % 3]
    W = _stack(torch, experts, rows, cols, scales, fp4=m % 2 == 0)
    off = _counts(kind, experts, m)
    x = torch.randn((m, cols), device="cuda").bfloat16()
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    y = nf4.nf4_expert_gemm(W, experts, x, offsets)
    ref, mag = _reference(torch, W, experts, x, off)
    _check(y, ref, mag, cols)


@pytest.mark.parametrize("experts,rows,cols,m", [s for s in SHAPES if s[1] % 8 == 0])
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_expert_gemm_dx(experts, rows, cols, m, kind):
    torch = need_gpu()
    say("expert dx", experts, rows, cols, m, kind)
    scales = ["int8", "fp8", "plain"][(rows + m) % 3]
    W = _stack(torch, experts, rows, cols, scales, fp4=m % 2 == 0)
    off = _counts(kind, experts, m)
    dy = torch.randn((m, rows), device="cuda").bfloat16()
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    dx = nf4.nf4_expert_gemm_dx(W, experts, dy, offsets)
    ref, mag = _reference(torch, W, experts, dy, off, dx=True)
    _check(dx, ref, mag, rows)


def _expert(W, experts, e):
    """Expert e of a stack with plain scales, on its own."""
    rows = W.rows // experts
    n = rows * W.cols
    return nf4.NF4Weight(W.packed[e * n // 2:(e + 1) * n // 2], rows, W.cols, absmax=W.absmax[e * n // 64:(e + 1) * n // 64])


def test_many_rows_equal_the_dense_product():
    """Experts of many rows: bit for bit nf4_gemm on each expert's rows (the
    same tiles and the same order of the sums)."""
    torch = need_gpu()
    experts, rows, cols, m = 3, 512, 768, 1500
    W = _stack(torch, experts, rows, cols, "plain")
    off = np.array([0, 700, 700, 1500])
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    x = torch.randn((m, cols), device="cuda").bfloat16()
    y = nf4.nf4_expert_gemm(W, experts, x, offsets)
    for e in (0, 2):
        at = slice(off[e], off[e + 1])
        assert torch.equal(y[at], nf4.nf4_gemm(_expert(W, experts, e), x[at]))


@pytest.mark.parametrize("experts,rows,cols,m", [
    (3, 64, 4096, 4200),      # a little over one round of whole tiles
    (3, 72, 4096, 6300),      # one round and a half
    (2, 40, 4160, 7700),      # a last round nearly full
    (70, 8, 1024, 18500),     # more experts than lanes of a wave
    (1, 256, 256, 300),       # whole tiles, but far from a round
])
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_dx_of_many_rows(experts, rows, cols, m, kind):
    """Sizes where two kernels share the gradient's rows: every row right, rows
    of no expert left alone, the same bits again."""
    torch = need_gpu()
    say("expert dx of many rows", experts, rows, cols, m, kind)
    W = _stack(torch, experts, rows, cols, "fp8")
    off = _counts(kind, experts, m - 2) + 1
    dy = torch.randn((m, rows), device="cuda").bfloat16()
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    dx = torch.full((m, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    nf4.nf4_expert_gemm_dx(W, experts, dy, offsets, dx=dx)
    assert (dx[0] == 7).all() and (dx[m - 1] == 7).all()
    ref, mag = _reference(torch, W, experts, dy, off, dx=True)
    _check(dx[1:m - 1], ref, mag, rows)
    assert torch.equal(dx[1:m - 1], nf4.nf4_expert_gemm_dx(W, experts, dy, offsets)[1:m - 1])


@pytest.mark.parametrize("experts,rows,cols,m", [
    (3, 4096, 64, 4200),      # a little over one round of 256-row tiles
    (2, 4090, 128, 7700),     # a last round nearly full
    (70, 1000, 64, 18500),    # more experts than lanes of a wave
    (1, 17, 64, 300),         # far from a round
])
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_gemm_of_many_rows(experts, rows, cols, m, kind):
    """Sizes where two launches share the product's rows."""
    torch = need_gpu()
    say("expert gemm of many rows", experts, rows, cols, m, kind)
    W = _stack(torch, experts, rows, cols, "fp8")
    off = _counts(kind, experts, m - 2) + 1
    x = torch.randn((200, cols), device="cuda").bfloat16()
    index = torch.randint(0, 400, (m,), device="cuda", dtype=torch.int32)
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    y = torch.full((m, rows), 7.0, dtype=torch.bfloat16, device="cuda")
    nf4.nf4_expert_gemm(W, experts, x, offsets, index=index, slots=2, y=y)
    assert (y[0] == 7).all() and (y[m - 1] == 7).all()
    ref, mag = _reference(torch, W, experts, x[(index // 2).long()], off)
    _check(y[1:m - 1], ref, mag, cols)


@pytest.mark.parametrize("mean", [10, 41, 113, 230])
def test_every_tile_height(mean):
    """The forward's kernels by the mean number of rows, one expert with most of them."""
    torch = need_gpu()
    experts, rows, cols = 5, 272, 192
    m = mean * experts
    W = _stack(torch, experts, rows, cols, "plain", fp4=True)
    c = np.array([0, m // 2, 1, 0, m - m // 2 - 1])
    off = np.concatenate([[0], np.cumsum(c)])
    x = torch.randn((m, cols), device="cuda").bfloat16()
    y = nf4.nf4_expert_gemm(W, experts, x, torch.from_numpy(off.astype(np.int32)).cuda())
    ref, mag = _reference(torch, W, experts, x, off)
    _check(y, ref, mag, cols)


@pytest.mark.parametrize("m", [6, 400])
def test_rows_of_no_expert_are_left(m):
    torch = need_gpu()
    experts, rows, cols = 4, 64, 128
    W = _stack(torch, experts, rows, cols)
    x = torch.randn((m, cols), device="cuda").bfloat16()
    dy = torch.randn((m, rows), device="cuda").bfloat16()
    off = np.array([1, 2, 2, m - 3, m - 2])
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    y = torch.full((m, rows), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((m, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    nf4.nf4_expert_gemm(W, experts, x, offsets, y=y)
    nf4.nf4_expert_gemm_dx(W, experts, dy, offsets, dx=dx)
    for out in (y, dx):
        assert (out[:1] == 7).all() and (out[m - 2:] == 7).all()
        assert not (out[1:m - 2] == 7).all(1).any()
    ref, mag = _reference(torch, W, experts, x, off)
    _check(y[1:m - 2], ref, mag, cols)
    # offsets that say nothing at all
    nf4.nf4_expert_gemm(W, experts, x, torch.zeros_like(offsets), y=y.fill_(7))
    assert (y == 7).all()


@pytest.mark.parametrize("m", [5, 300])
def test_offsets_and_indexes_out_of_range_stay_inside(m):
    """Clamped as documented: nothing outside the buffers is touched and the
    rows that the clamped offsets name are right."""
    torch = need_gpu()
    experts, rows, cols = 3, 32, 128
    W = _stack(torch, experts, rows, cols)
    x = torch.randn((m, cols), device="cuda").bfloat16()
    offsets = torch.tensor([-7, 2, 1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")  # expert 0: 0..1, 1: none, 2: 1..m-1
    index = torch.arange(m, dtype=torch.int32, device="cuda")
    index[-1] = 2 ** 31 - 1  # the last row of x
    index[0] = -2 ** 31      # the first
    y = nf4.nf4_expert_gemm(W, experts, x, torch.tensor([-7, 2, 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), index=index)
    ref, mag = _reference(torch, W, experts, x, [0, 2, 2, m])
    _check(y, ref, mag, cols)
    nf4.nf4_expert_gemm(W, experts, x, offsets)
    nf4.nf4_expert_gemm_dx(W, experts, torch.randn((m, rows), device="cuda").bfloat16(), offsets)
    torch.cuda.synchronize()


@pytest.mark.parametrize("tokens,slots,experts", [(1, 1, 1), (1, 2, 8), (9, 4, 16), (200, 2, 3)])
def test_gathered_rows(tokens, slots, experts):
    """index and slots give the rows that a sorted copy of x would hold, bit for bit."""
    torch = need_gpu()
    rows, cols = 96, 320
    W = _stack(torch, experts, rows, cols, "fp8")
    x = torch.randn((tokens, cols), device="cuda").bfloat16()
    ids = torch.rand((tokens, experts), device="cuda").topk(slots).indices.to(torch.int32)
    order, position, offsets = nf4.nf4_expert_plan(ids, experts)
    y = nf4.nf4_expert_gemm(W, experts, x, offsets, index=order, slots=slots)
    assert torch.equal(y, nf4.nf4_expert_gemm(W, experts, x[(order // slots).long()], offsets))


# ------------------------------------------------------------------- combine

def _positions(torch, tokens, slots, dropped, seed=4):
    g = np.random.default_rng(seed)
    n = tokens * slots
    p = g.permutation(n)
    p[g.random(n) < dropped] = -1
    return torch.from_numpy(p.reshape(tokens, slots).astype(np.int32)).cuda()


@pytest.mark.parametrize("tokens,slots,cols", [(1, 1, 8), (3, 2, 64), (7, 8, 40), (50, 3, 2048), (5, 2, 2056), (20, 1, 8200)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(tokens, slots, cols, weighted):
    """Forward: a float32 sum of `slots` products (each off by 2^-24, and each
    addition) and one rounding; backward: dy one rounding of one product,
    dweights a float32 sum of cols products."""
    torch = need_gpu()
    n = tokens * slots
    pos = _positions(torch, tokens, slots, 0.3)
    y = torch.randn((n, cols), device="cuda").bfloat16()
    wt = torch.rand((tokens, slots), device="cuda") if weighted else None
    out = nf4.nf4_expert_combine(y, pos, slots, weights=wt)
    live = (pos >= 0).double()[..., None]
    rows = y.double()[pos.clamp(min=0).long()] * live
    w64 = (wt.double() if weighted else torch.ones((tokens, slots), device="cuda", dtype=torch.float64))[..., None]
    ref, mag = (rows * w64).sum(1), (rows * w64).abs().sum(1)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2 * slots * 2.0 ** -24 * mag).all()
    dout = torch.randn((tokens, cols), device="cuda").bfloat16()
    dy = torch.full((n, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    dy2, dw = nf4.nf4_expert_combine_backward(dout, y, pos, slots, wt, dy=dy)
    assert dy2.data_ptr() == dy.data_ptr()
    want = torch.full_like(dy, 7.0)
    grads = ((wt[..., None] if weighted else 1.0) * dout.float()[:, None, :].expand(tokens, slots, cols)).to(torch.bfloat16)
    keep = pos.flatten() >= 0
    want[pos.flatten()[keep].long()] = grads.reshape(n, cols)[keep]
    assert torch.equal(dy, want)
    dref = (rows * dout.double()[:, None, :]).sum(-1)
    dmag = (rows * dout.double()[:, None, :]).abs().sum(-1)
    assert ((dw.double() - dref).abs() <= cols * 2.0 ** -24 * dmag).all()
    only, none = nf4.nf4_expert_combine_backward(dout, y, pos, slots, wt, dy=torch.full_like(dy, 7.0), want=("dy",))
    assert none is None and torch.equal(only, want)
    none, only = nf4.nf4_expert_combine_backward(dout, y, pos, slots, wt, want=("dweights",))
    assert none is None and torch.equal(only, dw)


def test_combine_positions_out_of_range_add_nothing():
    torch = need_gpu()
    y = torch.randn((4, 64), device="cuda").bfloat16()
    pos = torch.tensor([[0, 4], [2 ** 31 - 1, -2 ** 31], [3, 1]], dtype=torch.int32, device="cuda")
    out = nf4.nf4_expert_combine(y, pos, 2)
    assert torch.equal(out[0], y[0]) and (out[1] == 0).all()
    assert torch.equal(out[2], (y[3].float() + y[1].float()).bfloat16())
    dy, dw = nf4.nf4_expert_combine_backward(out, y, pos, 2, dy=torch.zeros_like(y))
    assert (dy[2] == 0).all() and dw[0, 1] == 0 and (dw[1] == 0).all()


# --------------------------------------------------------------- a whole layer

def _layer(torch, up, down, experts, x, ids, gate, dout):
    """One mixture-of-experts layer, forward and backward: two products with a
    product of halves between them."""
    slots = ids.shape[1]
    order, position, offsets = nf4.nf4_expert_plan(ids, experts)
    h = nf4.nf4_expert_gemm(up, experts, x, offsets, index=order, slots=slots)
    a, b = h.chunk(2, dim=1)
    z = (a * b).contiguous()
    o = nf4.nf4_expert_gemm(down, experts, z, offsets)
    out = nf4.nf4_expert_combine(o, position, slots, weights=gate)
    do, dgate = nf4.nf4_expert_combine_backward(dout, o, position, slots, gate)
    dz = nf4.nf4_expert_gemm_dx(down, experts, do, offsets)
    dh = torch.cat([dz * b, dz * a], dim=1)
    dxs = nf4.nf4_expert_gemm_dx(up, experts, dh, offsets)
    dx = nf4.nf4_expert_combine(dxs, position, slots)
    return out, dx, dgate


def _layer_ref(torch, up, down, experts, x, ids, gate, dout):
    """The same in float64 from dequantized weights, by autograd."""
    wu = nf4.nf4_dequantize(up, out_dtype=torch.float32).double().view(experts, -1, up.cols)
    wd = nf4.nf4_dequantize(down, out_dtype=torch.float32).double().view(experts, -1, down.cols)
    x, gate = x.double().requires_grad_(), gate.double().requires_grad_()
    out, size = torch.zeros_like(x), torch.zeros_like(gate)
    for e in range(experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        if len(t):
            a, b = (x[t] @ wu[e].t()).chunk(2, dim=1)
            o = (a * b) @ wd[e].t()
            out = out.index_add(0, t, o * gate[t, j][:, None])
            size = size.index_put((t, j), o.norm(dim=1))
    out.backward(dout.double())
    return (out.detach(), x.grad, gate.grad), size.detach()


@pytest.mark.parametrize("tokens", [2, 700])
def test_layer_forward_and_backward(tokens):
    """The operators together.  Nine roundings to bfloat16 (h, z, o, out; do, dz,
    dh, dx of the products, and their weights) of at most 2^-8 / sqrt(3) in the
    mean square each lie between the inputs and an output: sqrt(12) of them
    bound the relative error in the norm.  A gate's gradient <dout, o> can be
    small by cancellation: its error is at most |dout| times the error of o, and
    that is the same share of |o|."""
    torch = need_gpu()
    experts, slots, hidden, inner = 6, 2, 256, 192
    up, down = _stack(torch, experts, 2 * inner, hidden, "int8", seed=1), _stack(torch, experts, hidden, inner, "fp8", seed=2)
    x = torch.randn((tokens, hidden), device="cuda").bfloat16()
    ids = torch.rand((tokens, experts), device="cuda").topk(slots).indices.to(torch.int32)
    ids[0, 1] = -1  # a dropped slot
    gate = torch.rand((tokens, slots), device="cuda")
    dout = torch.randn((tokens, hidden), device="cuda").bfloat16()
    got = _layer(torch, up, down, experts, x, ids, gate, dout)
    ref, size = _layer_ref(torch, up, down, experts, x, ids, gate, dout)
    for g, r, scale in zip(got, ref, (ref[0], ref[1], size * dout.double().norm(dim=1)[:, None])):
        rel = ((g.double() - r).norm() / scale.norm()).item()
        assert rel <= 12 ** 0.5 * 2.0 ** -8 / 3 ** 0.5 * 1.5, rel
    assert got[2][0, 1] == 0


def test_layer_in_a_graph_follows_its_routing():
    """Captured once, replayed with other ids and activations: the eager
    results each time, with eager work between the replays."""
    torch = need_gpu()
    experts, slots, hidden, inner, tokens = 6, 2, 256, 192, 9
    up, down = _stack(torch, experts, 2 * inner, hidden, "int8", seed=1), _stack(torch, experts, hidden, inner, "plain", seed=2)
    x = torch.randn((tokens, hidden), device="cuda").bfloat16()
    ids = torch.rand((tokens, experts), device="cuda").topk(slots).indices.to(torch.int32)
    gate = torch.rand((tokens, slots), device="cuda")
    dout = torch.randn((tokens, hidden), device="cuda").bfloat16()
    _layer(torch, up, down, experts, x, ids, gate, dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        out = _layer(torch, up, down, experts, x, ids, gate, dout)
    for rep in range(4):
        x.copy_(torch.randn((tokens, hidden), device="cuda").bfloat16())
        new = torch.rand((tokens, experts), device="cuda").topk(slots).indices.to(torch.int32)
        if rep == 1:
            new[:] = 3           # everything to one expert
        ids.copy_(new)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, _layer(torch, up, down, experts, x, ids, gate, dout)):
            assert torch.equal(a, b), rep


def test_side_stream():
    """On a side stream with the binding's buffers, while the current stream
    allocates and fills memory: the results of the current stream."""
    torch = need_gpu()
    experts, slots, hidden, inner, tokens = 4, 2, 512, 256, 300
    W = _stack(torch, experts, inner, hidden)
    x = torch.randn((tokens, hidden), device="cuda").bfloat16()
    ids = torch.rand((tokens, experts), device="cuda").topk(slots).indices.to(torch.int32)

    def path(stream):
        order, position, offsets = nf4.nf4_expert_plan(ids, experts, stream=stream)
        y = nf4.nf4_expert_gemm(W, experts, x, offsets, index=order, slots=slots, stream=stream)
        dx = nf4.nf4_expert_gemm_dx(W, experts, y, offsets, stream=stream)
        return order, position, offsets, y, dx, nf4.nf4_expert_combine(dx, position, slots, stream=stream)

    ref = path(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = path(side)
    junk = [torch.full((t.numel() * t.element_size(),), 0xA5, dtype=torch.uint8, device="cuda") for t in ref for _ in range(3)]
    side.synchronize()
    torch.cuda.synchronize()
    del junk
    for a, b in zip(got, ref):
        assert torch.equal(a, b)


def test_weight_past_32_bit_offsets():
    """A stack of more than 2^32 weights: the last expert's are reached."""
    torch = need_gpu()
    experts, rows, cols = 33, 16384, 8192  # 4.4e9 weights, 2.2 GB of codes
    n = experts * rows * cols
    packed = torch.zeros(n // 2, dtype=torch.uint8, device="cuda").fill_(0x77)  # the zero level
    absmax = torch.ones(n // 64, device="cuda")
    last = (experts - 1) * rows * cols // 2
    packed[last:].random_(0, 256)
    W = nf4.NF4Weight(packed, experts * rows, cols, absmax=absmax)
    one = nf4.NF4Weight(packed[last:], rows, cols, absmax=absmax[:rows * cols // 64])
    x = torch.randn((3, cols), device="cuda").bfloat16()
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[experts - 1] = 1
    offsets[experts] = 3
    y = nf4.nf4_expert_gemm(W, experts, x, offsets)
    assert (y[0] == 0).all()
    w = nf4.nf4_dequantize(one, out_dtype=torch.float32).double()
    _check(y[1:], x[1:].double() @ w.t(), x[1:].double().abs() @ w.abs().t(), cols)
    dx = nf4.nf4_expert_gemm_dx(W, experts, y, offsets)
    assert (dx[0] == 0).all()
    _check(dx[1:], y[1:].double() @ w, y[1:].double().abs() @ w.abs(), rows)


@pytest.mark.parametrize("experts,m", [(6, 12), (6, 300), (4, 2000)])
def test_offsets_that_descend_stay_inside(experts, m):
    """All rows given to every other expert: a row gets some expert's product,
    and nothing around the outputs is touched."""
    torch = need_gpu()
    rows, cols, pad = 64, 128, 8
    W = _stack(torch, experts, rows, cols, "plain")
    offsets = torch.tensor([0, m] * (experts // 2) + [0], dtype=torch.int32, device="cuda")
    x = torch.randn((m, cols), device="cuda").bfloat16()
    dy = torch.randn((m, rows), device="cuda").bfloat16()
    y = torch.full((m + 2 * pad, rows), 7.0, dtype=torch.bfloat16, device="cuda")
    dx = torch.full((m + 2 * pad, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    nf4.nf4_expert_gemm(W, experts, x, offsets, y=y[pad:m + pad])
    nf4.nf4_expert_gemm_dx(W, experts, dy, offsets, dx=dx[pad:m + pad])
    for out in (y, dx):
        assert (out[:pad] == 7).all() and (out[m + pad:] == 7).all()
    each = [torch.tensor([0] * (e + 1) + [m] * (experts - e), dtype=torch.int32, device="cuda") for e in range(0, experts, 2)]
    ys = torch.stack([nf4.nf4_expert_gemm(W, experts, x, o) for o in each])
    assert (y[pad:m + pad] == ys).any(0).all()


@pytest.mark.parametrize("m", [16, 300, 1400])
def test_rows_stay_apart(m):
    """Infinities and NaN in one row of x or dy, and in rows of no expert, reach
    no other row."""
    torch = need_gpu()
    experts, rows, cols = 4, 256, 640
    W = _stack(torch, experts, rows, cols)
    off = np.array([3, 5, m // 2, m // 2, m - 4])
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    for call, k in ((nf4.nf4_expert_gemm, cols), (nf4.nf4_expert_gemm_dx, rows)):
        x = torch.randn((m, k), device="cuda").bfloat16()
        clean = call(W, experts, x, offsets)
        bad = [5, m - 6]
        x[bad[0], k // 2] = float("inf")
        x[bad[1]] = float("nan")
        x[:3] = float("nan")
        x[m - 4:] = float("nan")
        got = call(W, experts, x, offsets)
        good = torch.ones(m, dtype=torch.bool, device="cuda")
        good[bad] = False
        good[:3] = False
        good[m - 4:] = False
        assert torch.equal(got[good], clean[good])
        assert not got[bad].isfinite().any()


def test_dropped_slots_hide_what_is_not_finite():
    """NaN in a dropped slot's weight and in rows that no position names."""
    torch = need_gpu()
    tokens, slots, cols, m = 5, 3, 264, 20
    position = torch.arange(tokens * slots, dtype=torch.int32, device="cuda").view(tokens, slots)
    y = torch.randn((m, cols), device="cuda").bfloat16()
    weights = torch.rand((tokens, slots), device="cuda")
    dout = torch.randn((tokens, cols), device="cuda").bfloat16()
    position[1, 2], position[3, 0], position[4] = -1, m, -5
    dropped = (position < 0) | (position >= m)
    y[15:] = float("nan")
    y[[5, 9]] = float("nan")
    weights[dropped] = float("nan")
    out = nf4.nf4_expert_combine(y, position, slots, weights)
    dy, dweights = nf4.nf4_expert_combine_backward(dout, y, position, slots, weights, dy=torch.full_like(y, 7.0))
    assert out.isfinite().all() and (out[4] == 0).all()
    assert dweights.isfinite().all() and (dweights[dropped] == 0).all()
    named = torch.zeros(m, dtype=torch.bool, device="cuda")
    named[position[~dropped].long()] = True
    assert dy[named].isfinite().all() and (dy[~named] == 7).all()


def test_combine_of_more_slots_than_one_grid_dimension_counts():
    """2^26 slots and a few: one wave each in the backward sum is more than 2^32
    threads.  A gate's gradient is a float32 sum of 8 products, in any order: 8
    products and 7 additions, each off by 2^-24."""
    torch = need_gpu()
    n, cols, tail = 2 ** 26 + 5, 8, 1000
    position = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = torch.randn((n, cols), dtype=torch.bfloat16, device="cuda")
    dout = torch.randn((n, cols), dtype=torch.bfloat16, device="cuda")
    weights = torch.rand(n, device="cuda")
    out = nf4.nf4_expert_combine(y, position, 1, weights)
    dy, dweights = nf4.nf4_expert_combine_backward(dout, y, position, 1, weights)
    for at in (slice(0, tail), slice(n // 2, n // 2 + tail), slice(n - tail, n)):
        rows, w = position[at].long(), weights[at, None]
        assert torch.equal(out[at], (w * y[rows].float()).bfloat16())
        assert torch.equal(dy[rows], (w * dout[at].float()).bfloat16())
        p = dout[at].double() * y[rows].double()
        assert ((dweights[at, 0].double() - p.sum(1)).abs() <= 15 * 2.0 ** -24 * p.abs().sum(1) + 1e-30).all()


@pytest.mark.parametrize("experts,rows,cols,m", [
    (300, 8, 576, 700), (70, 40, 2112, 900), (16, 200, 4160, 640), (64, 1032, 1088, 3000), (9, 64, 8192, 500),  # 64-row tiles
    (20, 72, 1600, 3000), (9, 520, 2368, 1500), (4, 1000, 8128, 600),                                        # 128-row tiles
    (3, 136, 4096, 4200), (1, 56, 16384, 1030),                                                            # 256- and 64-row tiles
])
@pytest.mark.parametrize("kind", ["even", "one", "uneven"])
def test_dx_of_every_tile_height(experts, rows, cols, m, kind):
    """Reductions that end inside a step, columns that end inside a tile, each
    form of the scales; rows of no expert left, the same bits again."""
    torch = need_gpu()
    say("expert dx by tile height", experts, rows, cols, m, kind)
    for i, scales in enumerate(("int8", "fp8", "plain")):
        W = _stack(torch, experts, rows, cols, scales, fp4=(m + i) % 2 == 0)
        off = _counts(kind, experts, m - 2) + 1
        dy = torch.randn((m, rows), device="cuda").bfloat16()
        offsets = torch.from_numpy(off.astype(np.int32)).cuda()
        dx = torch.full((m, cols), 7.0, dtype=torch.bfloat16, device="cuda")
        nf4.nf4_expert_gemm_dx(W, experts, dy, offsets, dx=dx)
        assert (dx[0] == 7).all() and (dx[m - 1] == 7).all()
        ref, mag = _reference(torch, W, experts, dy, off, dx=True)
        _check(dx[1:m - 1], ref, mag, rows)
        assert torch.equal(dx[1:m - 1], nf4.nf4_expert_gemm_dx(W, experts, dy, offsets)[1:m - 1])


def test_dx_of_one_hot_rows_is_the_weight():
    """dy of ones in single places: the rows of the weight, rounded once to
    bfloat16, in every place of a step and of a tile."""
    torch = need_gpu()
    experts, rows, cols = 5, 200, 8256
    W = _stack(torch, experts, rows, cols, "fp8")
    m = experts * rows
    dy = torch.eye(rows, device="cuda").bfloat16().repeat(experts, 1)
    offsets = torch.arange(experts + 1, dtype=torch.int32, device="cuda") * rows
    assert torch.equal(nf4.nf4_expert_gemm_dx(W, experts, dy, offsets), nf4.nf4_dequantize(W, out_dtype=torch.float32).bfloat16())
    # many small experts: 64-row tiles
    small = 8
    one = torch.eye(small, device="cuda").bfloat16().repeat(m // small, 1)
    offsets = torch.arange(m // small + 1, dtype=torch.int32, device="cuda") * small
    assert torch.equal(nf4.nf4_expert_gemm_dx(W, m // small, one, offsets), nf4.nf4_dequantize(W, out_dtype=torch.float32).bfloat16())


def test_dx_of_a_weight_past_32_bit_offsets():
    """As above for products of whole tiles: the last expert's weights and scales."""
    torch = need_gpu()
    experts, rows, cols, m = 33, 16384, 8192, 600
    n = experts * rows * cols
    packed = torch.zeros(n // 2, dtype=torch.uint8, device="cuda").fill_(0x77)
    absmax = torch.ones(n // 64, device="cuda")
    last = (experts - 1) * rows * cols
    packed[last // 2:].random_(0, 256)
    absmax[last // 64:] = torch.rand(rows * cols // 64, device="cuda") + 0.5
    W = nf4.NF4Weight(packed, experts * rows, cols, absmax=absmax)
    one = nf4.NF4Weight(packed[last // 2:], rows, cols, absmax=absmax[last // 64:])
    dy = torch.randn((m, rows), device="cuda").bfloat16()
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device="cuda")
    offsets[experts - 1:] = torch.tensor([100, m], dtype=torch.int32)
    dx = nf4.nf4_expert_gemm_dx(W, experts, dy, offsets)
    assert (dx[:100] == 0).all()
    w = nf4.nf4_dequantize(one, out_dtype=torch.float32).double()
    d = dy[100:].double()
    _check(dx[100:], d @ w, d.abs() @ w.abs(), rows)
