"""nf4_linear against float64: every number of rows, activation, scale form and
argument that may be left out.

Bounds.  The weight enters the products in one of two readings (for a whole
call): rounded once to bf16 after scaling, which the reference then takes too,
or as the product of a level and a scale each rounded to fp16, rounded to fp16, off by
3 2^-11 of each weight at most (levels alone in fp16: 2^-11).  Sums of K
products in float32: K 2^-24 of the sum of magnitudes.  The adapters' thin
factor is summed in float32 and carried as two bf16 parts: 2^-16.  The
activation's slope is at most 1.13, its own evaluation good to 2^-16 of the
result (the exponential's argument, up to 88 in size, has 24 bits).  Then one
rounding to bf16."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.layer_common import ACTS, F32, HALF, SLOPE_MOST, act64, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(31)


def weight(torch, rows, cols, scales="int8", fp4=False):
    w = (torch.randn((rows, cols), device="cuda") / cols ** 0.5).bfloat16()
    return nf4.quantize_weight(w, double_quant=scales != "plain", dq_type="fp8" if scales == "fp8" else "int8",
                               quant_type="fp4" if fp4 else "nf4")


def check(torch, W, x, kw, y, pre=None, label=""):
    """y (and pre) of nf4_linear(W, x, **kw) within the bounds above, in one of the two readings."""
    xd = x.double().reshape(-1, W.cols)
    dense = {"bf16": nf4.nf4_dequantize(W, out_dtype=torch.bfloat16).double(), "levels": nf4.nf4_dequantize(W, out_dtype=torch.float32).double()}
    terms = W.cols + 8
    res, act = kw.get("residual"), kw.get("act", "none")
    found = {}
    for reading, wd in dense.items():
        z = xd @ wd.t()
        err = (terms * F32 + (3 * 2.0 ** -11 if reading == "levels" else 0.0)) * (xd.abs() @ wd.abs().t())
        if kw.get("lora_a") is not None:
            a, b, s = kw["lora_a"].double(), kw["lora_b"].double(), kw["lora_scale"]
            z = z + s * (xd @ a.t()) @ b.t()
            err = err + (2.0 ** -16 + (terms + a.shape[0]) * F32) * abs(s) * (xd.abs() @ a.abs().t()) @ b.abs().t()
        if kw.get("bias") is not None:
            z = z + kw["bias"].double()
        err = err + 4 * F32 * z.abs()
        v = act64(torch, act, z)
        out = v + res.double().reshape(z.shape) if res is not None else v
        off = SLOPE_MOST * err + 2.0 ** -16 * v.abs() + 1e-35
        off = HALF["bf16"] * (out.abs() + off) + off
        shares = [worst((y.double() - out).abs(), off)]
        if pre is not None:
            shares.append(worst((pre.double() - z).abs(), HALF["bf16"] * (z.abs() + err) + err + 1e-35))
        found[reading] = max(shares)
    say(f"  {label} worst element over its bound: {found}")
    assert min(found.values()) <= 1.0, found


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


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 8, 15, 16, 17, 31, 32, 33, 40, 63, 64, 65, 96, 127, 128, 129, 200, 255, 257, 513])
@pytest.mark.parametrize("rows,cols", [(384, 1024), (200, 576)])
def test_rows_of_x(m, rows, cols):
    torch = need_gpu()
    say("linear", m, rows, cols)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16", residual=True)
    y, pre = nf4.nf4_linear(W, x, act="silu", save_pre=True, **kw)
    check(torch, W, x, dict(kw, act="silu"), y, pre, f"m {m}")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [1, 3, 16, 50, 300])
def test_activations(act, m):
    torch = need_gpu()
    say("linear", act, m)
    rows, cols = 264, 512
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "f32")
    x = x * 3  # into the tails
    y, pre = nf4.nf4_linear(W, x, act=act, save_pre=True, **kw)
    check(torch, W, x, dict(kw, act=act), y, pre, act)


@pytest.mark.parametrize("scales,fp4", [("plain", False), ("int8", False), ("fp8", False), ("int8", True), ("plain", True)])
@pytest.mark.parametrize("m", [1, 2, 9, 70, 260])
def test_scale_forms(scales, fp4, m):
    torch = need_gpu()
    say("linear", scales, fp4, m)
    rows, cols = 320, 1088
    W = weight(torch, rows, cols, scales, fp4)
    x, kw = inputs(torch, m, rows, cols, "bf16")
    check(torch, W, x, dict(kw, act="gelu"), nf4.nf4_linear(W, x, act="gelu", **kw), label=scales)


# rows that end inside every tile, from one on; widths of one block and of many odd ones
@pytest.mark.parametrize("rows,cols", [(1, 64), (2, 64), (7, 128), (15, 192), (17, 64), (33, 448), (63, 4160), (65, 64), (129, 320),
                                       (255, 64), (257, 64), (511, 128), (1000, 64), (31, 9024), (5, 14336)])
@pytest.mark.parametrize("m", [1, 4, 13, 16, 37, 100, 258])
def test_ragged(rows, cols, m):
    torch = need_gpu()
    say("linear", rows, cols, m)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "f32", residual=True, rank=3)
    y, pre = nf4.nf4_linear(W, x, act="gelu_tanh", save_pre=True, **kw)
    check(torch, W, x, dict(kw, act="gelu_tanh"), y, pre)


@pytest.mark.parametrize("rank", [1, 7, 16, 17, 32, 48, 64])
@pytest.mark.parametrize("m", [1, 2, 16, 48, 130])
def test_adapters(rank, m):
    torch = need_gpu()
    say("linear adapters", rank, m)
    rows, cols = 328, 640
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16", rank=rank)
    y = nf4.nf4_linear(W, x, act="relu", **kw)
    check(torch, W, x, dict(kw, act="relu"), y)
    # B of zeros adds nothing at all
    zero = dict(kw, lora_b=torch.zeros_like(kw["lora_b"]))
    bare = {k: v for k, v in kw.items() if not k.startswith("lora")}
    assert torch.equal(nf4.nf4_linear(W, x, **zero), nf4.nf4_linear(W, x, **bare))


@pytest.mark.parametrize("m", [1, 2, 7, 16, 60, 129, 300])
def test_what_may_be_left_out(m):
    """Nothing in the epilogue: the bare product; each argument alone."""
    torch = need_gpu()
    say("linear arguments", m)
    rows, cols = 256, 768
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16", residual=True, rank=8)
    for keys in ((), ("bias",), ("residual",), ("lora_a", "lora_b", "lora_scale"), ("bias", "residual")):
        part = {k: kw[k] for k in keys}
        check(torch, W, x, part, nf4.nf4_linear(W, x, **part), label=str(keys))
    y, pre = nf4.nf4_linear(W, x, save_pre=True)
    assert torch.equal(y, pre)  # without an activation and a residual


@pytest.mark.parametrize("m", [1, 3, 16, 33, 90, 280])
def test_buffers_of_the_caller(m):
    """The residual added in place, given outputs and workspace, rows outside left alone."""
    torch = need_gpu()
    say("linear buffers", m)
    rows, cols = 203, 512
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "f32", residual=True, rank=5)
    want, want_pre = nf4.nf4_linear(W, x, act="silu", save_pre=True, **kw)
    room = torch.full((2, m * rows + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    y, pre = room[0, :m * rows], torch.full((m * rows + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
    y.copy_(kw["residual"].reshape(-1))
    ws = torch.full((nf4.nf4_linear_workspace(m, rows, cols, 5),), 255, dtype=torch.uint8, device="cuda")
    got = nf4.nf4_linear(W, x, act="silu", **dict(kw, residual=y), y=y, pre=pre[:m * rows], workspace=ws)
    assert got[0].data_ptr() == y.data_ptr() and got[1].data_ptr() == pre.data_ptr()
    assert torch.equal(y.view(m, rows), want) and torch.equal(pre[:m * rows].view(m, rows), want_pre)
    assert (room[0, m * rows:] == 7).all() and (room[1] == 7).all() and (pre[m * rows:] == 7).all()


@pytest.mark.parametrize("m", [1, 8, 40, 140, 520])
def test_same_twice_and_rows_apart(m):
    """Deterministic; a row of x that is not finite reaches no other row."""
    torch = need_gpu()
    say("linear rows apart", m)
    rows, cols = 336, 2112
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16", residual=True, rank=4)
    y = nf4.nf4_linear(W, x, act="gelu", **kw)
    assert torch.equal(y, nf4.nf4_linear(W, x, act="gelu", **kw))
    if m > 1:
        bad = x.clone()
        bad[m // 2] = float("nan")
        z = nf4.nf4_linear(W, bad, act="gelu", **kw)
        keep = torch.arange(m, device="cuda") != m // 2
        assert torch.equal(z[keep], y[keep]) and z[m // 2].isnan().all()


# one or two rows of wide and of many-rowed weights; a decode batch over one and many groups of weight rows per
# workgroup, one and many column segments per wave; cut reductions; whole tiles
@pytest.mark.parametrize("m,rows,cols", [
    (1, 1003, 4160), (2, 1003, 4160), (1, 12301, 704), (2, 12301, 704), (1, 40, 33024), (2, 40, 33024), (1, 3, 66048), (2, 9, 66048),
    (3, 14343, 640), (16, 14343, 640), (7, 20001, 448), (3, 70001, 64), (5, 300007, 64), (11, 9001, 4416), (6, 24013, 4416),
    (4, 24013, 1088), (2, 33, 14400), (13, 5, 33024), (9, 4099, 14400),
    (20, 9001, 320), (37, 4099, 576), (49, 2000, 2112), (700, 33, 1088), (1100, 70, 320), (2050, 16, 64), (4100, 3, 128),
    (17, 9001, 4416), (40, 9001, 4416), (150, 2001, 4160), (330, 2001, 4160), (600, 1999, 4160), (1000, 1003, 3648), (97, 8199, 2112), (1300, 259, 2112),
    (300, 9007, 640), (700, 9007, 640), (513, 7001, 1088), (2500, 515, 1088), (400, 14343, 192), (5000, 70, 192)])
def test_sizes_of_every_kernel(m, rows, cols):
    torch = need_gpu()
    say("linear sizes", m, rows, cols)
    W = weight(torch, rows, cols, ("int8", "fp8", "plain")[(m + rows) % 3], fp4=m % 5 == 0)
    x, kw = inputs(torch, m, rows, cols, "f32", residual=True, rank=(m % 4) * 5)
    y, pre = nf4.nf4_linear(W, x, act="gelu", save_pre=True, **kw)
    check(torch, W, x, dict(kw, act="gelu"), y, pre)
    assert torch.equal(y, nf4.nf4_linear(W, x, act="gelu", **kw))


# sizes of the kernel that cuts the reduction, with and without a second launch to join it, and of whole tiles
LARGER = [(330, 2001, 4160), (520, 4001, 2112), (700, 9007, 640), (2100, 4100, 192)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,rows,cols", LARGER)
def test_activations_of_larger_sizes(act, m, rows, cols):
    torch = need_gpu()
    say("linear", act, m, rows, cols)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16", residual=True)
    x = x * 3
    y, pre = nf4.nf4_linear(W, x, act=act, save_pre=True, **kw)
    check(torch, W, x, dict(kw, act=act), y, pre, act)


@pytest.mark.parametrize("scales,fp4", [("plain", False), ("int8", False), ("fp8", False), ("int8", True), ("fp8", True), ("plain", True)])
@pytest.mark.parametrize("m,rows,cols", LARGER)
def test_scale_forms_of_larger_sizes(scales, fp4, m, rows, cols):
    torch = need_gpu()
    say("linear", scales, fp4, m, rows, cols)
    W = weight(torch, rows, cols, scales, fp4)
    x, kw = inputs(torch, m, rows, cols)
    check(torch, W, x, kw, nf4.nf4_linear(W, x), label=scales)


@pytest.mark.parametrize("rank", [1, 7, 16, 17, 48, 64])
@pytest.mark.parametrize("m,rows,cols", LARGER + [(3, 1000, 5184), (1, 1000, 5184), (200, 515, 576)])
def test_adapters_of_larger_sizes(rank, m, rows, cols):
    torch = need_gpu()
    say("linear adapters", rank, m, rows, cols)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "f32", rank=rank)
    check(torch, W, x, kw, nf4.nf4_linear(W, x, **kw))
    zero = dict(kw, lora_b=torch.zeros_like(kw["lora_b"]))
    assert torch.equal(nf4.nf4_linear(W, x, **zero), nf4.nf4_linear(W, x, bias=kw["bias"]))


@pytest.mark.parametrize("m,rows,cols", LARGER + [(2, 1001, 4160), (16, 9001, 4416)])
def test_buffers_and_rows_apart_of_larger_sizes(m, rows, cols):
    """The residual added in place, given outputs and workspace, rows outside left alone; a row that is not finite reaches no other."""
    torch = need_gpu()
    say("linear buffers", m, rows, cols)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "f32", residual=True, rank=5)
    want, want_pre = nf4.nf4_linear(W, x, act="silu", save_pre=True, **kw)
    y, pre = torch.full((2, m * rows + 64), 7.0, dtype=torch.bfloat16, device="cuda").unbind()
    pre = torch.full_like(pre, 7.0)
    y[:m * rows].copy_(kw["residual"].reshape(-1))
    ws = torch.full((nf4.nf4_linear_workspace(m, rows, cols, 5) + 256,), 255, dtype=torch.uint8, device="cuda")
    nf4.nf4_linear(W, x, act="silu", **dict(kw, residual=y[:m * rows]), y=y[:m * rows], pre=pre[:m * rows], workspace=ws[:-256])
    assert torch.equal(y[:m * rows].view(m, rows), want) and torch.equal(pre[:m * rows].view(m, rows), want_pre)
    assert (y[m * rows:] == 7).all() and (pre[m * rows:] == 7).all() and (ws[-256:] == 255).all()
    for value in (float("nan"), float("inf")):
        bad = x.clone()
        bad[m // 2, 3] = value
        z = nf4.nf4_linear(W, bad, act="silu", **kw)
        keep = torch.arange(m, device="cuda") != m // 2
        assert torch.equal(z[keep], want[keep])
        if value != value:
            assert z[m // 2].isnan().all()


@pytest.mark.parametrize("m,rows,cols", LARGER + [(1, 1001, 4160), (2, 1001, 4160), (9, 4099, 4160)])
@pytest.mark.parametrize("up,down", [(60, -50), (-60, 50), (90, -100), (-100, 90)])
def test_range_of_larger_sizes(m, rows, cols, up, down):
    """Weights and activations of any magnitude, whose products are ordinary numbers; rows of x of zeros."""
    torch = need_gpu()
    say("linear range", m, rows, cols, up)
    W = nf4.quantize_weight(torch.randn((rows, cols), device="cuda").bfloat16() * 2.0 ** up)
    x = (torch.randn((m, cols), device="cuda") * 2.0 ** down).bfloat16()
    x[m // 3] = 0
    check(torch, W, x, dict(act="silu"), nf4.nf4_linear(W, x, act="silu"))


@pytest.mark.parametrize("m,rows,cols", LARGER + [(2, 1001, 4160), (20, 9001, 4416)])
def test_graph_of_larger_sizes(m, rows, cols):
    """Captured once and replayed with other inputs, eager work between: each replay equals the eager call bit for bit."""
    torch = need_gpu()
    say("linear graph", m, rows, cols)
    W = weight(torch, rows, cols)
    x, kw = inputs(torch, m, rows, cols, "bf16", residual=True, rank=16)
    y, pre = (torch.empty((m, rows), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ws = torch.empty(nf4.nf4_linear_workspace(m, rows, cols, 16), dtype=torch.uint8, device="cuda")
    call = lambda y, pre: nf4.nf4_linear(W, x, act="gelu", y=y, pre=pre, workspace=ws, **kw)  # noqa: E731
    call(y, pre)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="relaxed"):
        call(y, pre)
    for rep in range(3):
        x.copy_(torch.randn_like(x))
        kw["residual"].copy_(torch.randn_like(kw["residual"]))
        want = [torch.empty_like(y) for _ in range(2)]
        call(*want)
        y.zero_()
        pre.zero_()
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(pre, want[1]), rep


def test_many_tiles():
    """More work units than compute units, the last round cut in halves, and widths of several column tiles."""
    torch = need_gpu()
    for m, rows, cols in ((1030, 4352, 256), (2500, 3400, 128), (4096, 8200, 64)):
        say("linear tiles", m, rows, cols)
        W = weight(torch, rows, cols)
        x, kw = inputs(torch, m, rows, cols, "f32", residual=True, rank=2)
        y, pre = nf4.nf4_linear(W, x, act="silu", save_pre=True, **kw)
        check(torch, W, x, dict(kw, act="silu"), y, pre)


def test_leading_dimensions_and_no_rows():
    torch = need_gpu()
    W = weight(torch, 96, 128)
    x = torch.randn((3, 5, 128), device="cuda").bfloat16()
    b = torch.randn(96, device="cuda")
    assert torch.equal(nf4.nf4_linear(W, x, bias=b), nf4.nf4_linear(W, x.reshape(15, 128), bias=b))
    assert torch.equal(nf4.nf4_linear(W, x.transpose(0, 1), bias=b), nf4.nf4_linear(W, x.transpose(0, 1).contiguous(), bias=b))
    y, pre = nf4.nf4_linear(W, x[:0], bias=b, act="gelu", save_pre=True)
    assert tuple(y.shape) == (0, 96) and tuple(pre.shape) == (0, 96)
    with pytest.raises(ValueError):
        nf4.nf4_linear(W, x[:0], bias=b[:-1])


@pytest.mark.parametrize("m", [1, 16, 64, 300])
def test_large_values(m):
    """Weights and activations near the ends of bf16's range: finite where the definition is."""
    torch = need_gpu()
    rows, cols = 64, 128
    w = torch.randn((rows, cols), device="cuda").bfloat16() * 2.0 ** 60
    W = nf4.quantize_weight(w)
    x = (torch.randn((m, cols), device="cuda") * 2.0 ** 50).bfloat16()
    check(torch, W, x, dict(act="silu"), nf4.nf4_linear(W, x, act="silu"))
    x = (torch.randn((m, cols), device="cuda") * 2.0 ** -70).bfloat16()
    check(torch, W, x, dict(act="gelu_tanh"), nf4.nf4_linear(W, x, act="gelu_tanh"))
