"""Uniform 4-bit weights with group scales on the GPU: quantizer and
dequantizer against a numpy float32 computation (bit for bit), the decode
product against float64.

Tolerance of the product, per output (S = sum |x| s over the row's columns):
half a step of the output's type on the value, plus the float32 sums.  A
group's operands 1 + q / 16 and its correction are at most 2 each, times 16 s,
so its terms add up to at most 64 |x| s; a sum of n terms in float32 is off by
at most n 2^-24 of the sum of their magnitudes, with n = group terms, then one
addition per group and wave and a few roundings of the scale and corrections:
(group + cols / group + 24) 2^-24 . 64 S."""

from __future__ import annotations

import numpy as np
import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(21)


def _types(torch):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _round_to(a, kind):
    """float32 values rounded to the type, as float32."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, np.float32))
    return t.to(_types(torch)[kind]).to(torch.float32).numpy()


def _quantize_np(w, group, asym, kind):
    """(codes, scales, zeros) by the definition, in float32."""
    x = np.ascontiguousarray(w, np.float32).reshape(w.shape[0], -1, group)
    one = np.float32
    if asym:
        lo, hi = np.minimum(x.min(-1), one(0)), np.maximum(x.max(-1), one(0))
        s = _round_to((hi - lo) / one(15), kind)
    else:
        s = _round_to(np.abs(x).max(-1) / one(7), kind)
    if kind == "f16":
        s = np.minimum(s, one(65504))
    by = np.where(s > 0, s, one(1))
    z = np.where(s > 0, np.clip(np.rint(-lo / by), 0, 15), 0) if asym else np.full_like(s, 8)
    q = np.clip(np.rint(x / by[..., None]) + z[..., None], 0, 15)
    q = np.where(s[..., None] > 0, q, z[..., None])
    return q.reshape(w.shape).astype(np.uint8), s, z.astype(np.uint8)


def _pack(q):
    q = q.reshape(-1)
    return (q[0::2] << 4) | q[1::2]


def _weights(torch, rows, cols, kind, seed):
    g = np.random.default_rng(seed)
    w = g.standard_normal((rows, cols)).astype(np.float32) * 0.02
    w[g.random((rows, cols)) < 0.002] *= 20
    w[0, :32] = 0.0  # a group (or a part of one) of zeros
    if rows > 1:
        w[1] = np.abs(w[1]) + 0.001  # one sign only
    if rows > 2:
        w[2] *= -np.sign(w[2])
    if rows > 3:
        w[3] = np.float32(1e-9)      # scales that vanish in float16
    if rows > 4:
        w[4] = w[4] * np.float32(1e-30)
    return torch.from_numpy(w).to(_types(torch)[kind])


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scale", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("asym", [False, True])
def test_int4_coding_bit_exact(kind, scale, group, asym):
    torch = need_gpu()
    rows, cols = 37, 384
    say("int4 coding", kind, scale, group, asym)
    w = _weights(torch, rows, cols, kind, 5)
    T = _types(torch)
    W = nf4.quantize_int4(w.cuda(), group=group, symmetric=not asym, scale_dtype=T[scale])
    q, s, z = _quantize_np(w.float().numpy(), group, asym, scale)
    assert np.array_equal(W.scales.float().cpu().numpy(), s)
    if asym:
        assert np.array_equal(W.zeros.cpu().numpy(), z)
    else:
        assert W.zeros is None
    assert np.array_equal(W.packed.cpu().numpy(), _pack(q))
    value = ((q.reshape(rows, -1, group).astype(np.float32) - z[..., None].astype(np.float32)) * s[..., None]).reshape(rows, cols)
    for out in T.values():
        got = nf4.nf4_int4_dequantize(W, out_dtype=out)
        assert torch.equal(got.cpu(), torch.from_numpy(value).to(out)), out


def test_int4_coding_rounds_ties_to_even_and_saturates():
    torch = need_gpu()
    # symmetric, max 7: the scale is exactly 1
    w = torch.zeros(2, 32)
    w[0, :8] = torch.tensor([7.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, -7.0])
    w[1, :4] = torch.tensor([3.0e6, -3.0e6, 1.0e6, 0.0])  # max / 7 is past float16's range
    W = nf4.quantize_int4(w.cuda(), group=32, scale_dtype=torch.float16)
    codes = W.packed.cpu().numpy()
    q = np.stack([codes >> 4, codes & 15], 1).reshape(2, 32)
    assert q[0, :8].tolist() == [15, 8, 10, 10, 8, 6, 6, 1]
    assert W.scales.cpu().flatten().tolist() == [1.0, 65504.0]
    assert q[1, :4].tolist() == [15, 0, 15, 8]


def _product(torch, rows, cols, group, asym, m, x_kind, scale, y_kind, seed):
    T = _types(torch)
    g = torch.Generator(device="cuda").manual_seed(seed)
    packed = torch.randint(0, 256, (rows * cols // 2,), generator=g, device="cuda", dtype=torch.uint8)
    shape = (rows, cols // group)
    scales = (0.001 + 0.02 * torch.rand(shape, generator=g, device="cuda")).to(T[scale])
    scales[torch.rand(shape, generator=g, device="cuda") < 0.1] = 0
    zeros = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8) if asym else None
    x = torch.randn((m, cols), generator=g, device="cuda").to(T[x_kind])
    W = nf4.Int4Weight(packed, rows, cols, group, scales, zeros)
    y = nf4.nf4_int4_gemv(W, x, y_dtype=T[y_kind])
    q = torch.stack((packed >> 4, packed & 15), 1).reshape(rows, -1, group).double()
    z = zeros.double()[..., None] if asym else 8.0
    ref = x.double() @ ((q - z) * scales.double()[..., None]).reshape(rows, cols).t()
    S = x.double().abs() @ scales.double().repeat_interleave(group, 1).t()
    return W, x, y, ref, S


def _check_product(torch, y, ref, S, group, cols):
    half = torch.finfo(y.dtype).eps / 2
    tiny = torch.finfo(y.dtype).smallest_normal * torch.finfo(y.dtype).eps  # half a step below the normal range
    bound = half * ref.abs() + (group + cols / group + 24) * 2.0 ** -24 * 64 * S + tiny
    worst = ((y.double() - ref).abs() / bound).max().item()
    assert worst <= 1.0, worst


@pytest.mark.parametrize("m", [1, 2, 3, 5, 8, 15, 16])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("asym", [False, True])
def test_int4_gemv_rows_of_x(m, group, asym):
    torch = need_gpu()
    say("int4 gemv", m, group, asym)
    for x_kind, scale, y_kind in (("bf16", "f16", "f32"), ("f16", "bf16", "bf16"), ("bf16", "f32", "f16")):
        _, _, y, ref, S = _product(torch, 83, 640, group, asym, m, x_kind, scale, y_kind, m)
        _check_product(torch, y, ref, S, group, 640)


@pytest.mark.parametrize("rows,cols,group", [
    (1, 32, 32), (1, 128, 128), (15, 96, 32), (16, 64, 64), (17, 192, 64), (4096, 128, 128), (5, 4096, 128),
    (300, 3584, 128), (33, 4128, 32), (70, 8256, 64), (257, 14336, 128), (40, 28672, 64), (19, 65536, 128), (9000, 256, 32),
])
@pytest.mark.parametrize("m", [1, 16])
def test_int4_gemv_shapes(rows, cols, group, m):
    torch = need_gpu()
    say("int4 gemv", rows, cols, group, m)
    _, _, y, ref, S = _product(torch, rows, cols, group, rows % 2 == 1, m, "bf16", "f16", "f32", rows + cols)
    _check_product(torch, y, ref, S, group, cols)
    rel = ((y.double() - ref).norm() / ref.norm()).item()
    assert rel <= 1e-5, rel


def test_int4_gemv_one_hot_returns_the_column():
    """x with a single 1 gives the dequantized column: exact in float32 but
    for the correction's two roundings (of values up to 64 s)."""
    torch = need_gpu()
    W, x, _, _, _ = _product(torch, 50, 512, 64, True, 4, "bf16", "bf16", "f32", 3)
    x.zero_()
    at = [0, 63, 257, 511]
    for i, c in enumerate(at):
        x[i, c] = 1
    y = nf4.nf4_int4_gemv(W, x, y_dtype=torch.float32)
    col = nf4.nf4_int4_dequantize(W, out_dtype=torch.float32)[:, at].t()
    s = W.scales.float()[:, [c // 64 for c in at]].t()
    assert ((y - col).abs() <= 64 * s * 2.0 ** -23).all()


def test_int4_gemv_repeats_bit_for_bit_and_leaves_neighbours():
    torch = need_gpu()
    W, x, y, _, _ = _product(torch, 1000, 2048, 128, True, 7, "bf16", "f16", "bf16", 9)
    out = torch.full((7 * 1000 + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        nf4.nf4_int4_gemv(W, x, y=out[:7000])
        assert torch.equal(out[:7000].view(7, 1000), y)
    assert (out[7000:] == 3).all()


def test_int4_graph_and_side_stream():
    """Quantizer and product captured into a graph and replayed on new inputs,
    and called on a side stream: the eager results, bit for bit."""
    torch = need_gpu()
    w = torch.randn(96, 512, device="cuda").bfloat16()
    x = torch.randn(3, 512, device="cuda").bfloat16()
    W = nf4.quantize_int4(w, group=64, symmetric=False)
    y = torch.empty(3, 96, device="cuda", dtype=torch.bfloat16)

    def path():
        nf4.nf4_int4_quantize(w, W)
        nf4.nf4_int4_gemv(W, x, y=y)

    path()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        path()
    for rep in range(3):
        w.copy_(torch.randn(96, 512, device="cuda").bfloat16())
        x.copy_(torch.randn(3, 512, device="cuda").bfloat16())
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        eager = nf4.nf4_int4_gemv(nf4.quantize_int4(w, group=64, symmetric=False), x)
        assert torch.equal(eager, y), rep
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nf4.nf4_int4_gemv(nf4.quantize_int4(w, group=64, symmetric=False, stream=side), x, stream=side)
    junk = [torch.full((w.numel() // 2,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(8)]
    side.synchronize()
    del junk
    assert torch.equal(got, y)


def test_int4_coding_of_more_blocks_than_one_grid_dimension():
    """A weight of more than 2^32 values: its first and last rows as if alone."""
    torch = need_gpu()
    rows, cols, few = 65600, 65536, 40
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    for at in (slice(0, few), slice(rows - few, rows)):
        x[at] = torch.randn((few, cols), device="cuda").bfloat16()
    W = nf4.quantize_int4(x, group=64, symmetric=False)
    out = nf4.nf4_int4_dequantize(W)
    for at in (slice(0, few), slice(rows - few, rows)):
        one = nf4.quantize_int4(x[at], group=64, symmetric=False)
        assert torch.equal(W.packed.view(rows, -1)[at], one.packed.view(few, -1))
        assert torch.equal(W.scales[at], one.scales) and torch.equal(W.zeros[at], one.zeros)
        assert torch.equal(out[at], nf4.nf4_int4_dequantize(one))
    assert not out[few:rows - few].any()
