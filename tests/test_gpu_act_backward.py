"""nf4_act_backward against float64 and against differences of the forward.

Bounds: the slope is formed in float32, off by at most 2^-16 (its exponential's
argument has 24 bits, and 1 - s loses 2^-24 times a factor below 40 where it
counts); one rounding of dz; sums of m terms in float32."""

from __future__ import annotations

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.layer_common import ACTS, F32, HALF, act64, slope64, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(37)


def check(torch, act, dy, pre, dz, dbias):
    d = dy.double()
    ref = d * slope64(torch, act, pre.double()) if act != "none" else d
    off = (0.0 if act == "none" else 2.0 ** -16) * d.abs() + 1e-38
    if dz is not None:
        share = worst((dz.double() - ref).abs(), HALF["bf16"] * (ref.abs() + off) + off)
        assert share <= 1.0, (act, "dz", share)
    if dbias is not None:
        m = dy.shape[0]
        share = worst((dbias.double() - ref.sum(0)).abs(), (off + m * F32 * (ref.abs() + off)).sum(0))
        assert share <= 1.0, (act, "dbias", share)


SIZES = [(1, 1), (1, 8), (3, 7), (1, 4097), (257, 1), (5, 9), (64, 64), (100, 2050), (33, 11007), (1000, 24), (4100, 130), (2, 28672),
         (700, 1024)]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,rows", SIZES)
def test_against_float64(act, m, rows):
    torch = need_gpu()
    say("act backward", act, m, rows)
    dy = torch.randn((m, rows), device="cuda").bfloat16()
    pre = (2.5 * torch.randn((m, rows), device="cuda")).bfloat16()
    dz, db = nf4.nf4_act_backward(dy, pre, act)
    check(torch, act, dy, pre, dz, db)
    # each alone, the same bits
    only, none = nf4.nf4_act_backward(dy, pre, act, want=("dz",))
    assert none is None and torch.equal(only, dz)
    none, only = nf4.nf4_act_backward(dy, pre, act, want=("dbias",))
    assert none is None and torch.equal(only, db)


@pytest.mark.parametrize("act", ACTS[1:])
def test_every_bf16(act):
    """The slope at every finite bf16 value, and at the infinities its limits."""
    torch = need_gpu()
    bits = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16)
    pre = bits.view(torch.bfloat16)
    pre = pre[pre.isfinite()].reshape(-1, 8)
    dy = torch.ones_like(pre)
    dz, _ = nf4.nf4_act_backward(dy, pre, act)
    wide = pre.double().clamp(-1e4, 1e4)  # where the formula in 64 bits itself overflows, the slope has its limit
    check(torch, act, dy, wide, dz, None)
    ends = torch.tensor([[float("inf"), -float("inf"), float("nan"), 0.0]], device="cuda").bfloat16()
    got, _ = nf4.nf4_act_backward(torch.ones_like(ends), ends, act, want=("dz",))
    assert got[0, 0] == 1 and got[0, 1] == 0 and got[0, 2].isnan() and got[0, 3] == (0.0 if act == "relu" else 0.5)


@pytest.mark.parametrize("act", ACTS[1:])
def test_against_differences(act):
    """The slope is the derivative of what nf4_linear applies: central differences of the 64-bit
    definition, step h: off by h^2 / 6 times the third derivative (below 4) and the slope's own 2^-16."""
    torch = need_gpu()
    pre = (torch.linspace(-6, 6, 4096, device="cuda").bfloat16() + 2.0 ** -9).bfloat16().reshape(8, -1)
    dz, _ = nf4.nf4_act_backward(torch.ones_like(pre), pre, act, want=("dz",))
    h, z = 1e-4, pre.double()
    if act == "relu":
        z = torch.where(z.abs() < 2 * h, torch.full_like(z, 1.0), z)
        dz = torch.where(pre.double().abs() < 2 * h, torch.ones_like(dz), dz)
    ref = (act64(torch, act, z + h) - act64(torch, act, z - h)) / (2 * h)
    assert worst((dz.double() - ref).abs(), HALF["bf16"] * ref.abs() + 2.0 ** -16 + 4 * h * h + 1e-10) <= 1.0


@pytest.mark.parametrize("m,rows", [(9, 13), (300, 520)])
def test_in_place_and_buffers(m, rows):
    torch = need_gpu()
    dy = torch.randn((m, rows), device="cuda").bfloat16()
    pre = torch.randn((m, rows), device="cuda").bfloat16()
    dz, db = nf4.nf4_act_backward(dy, pre, "gelu")
    room = torch.full((m * rows + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    mine = room[:m * rows].view(m, rows)
    mine.copy_(dy)
    bias = torch.full((rows + 4,), 7.0, device="cuda")
    ws = torch.full((max(1, nf4.nf4_act_backward_workspace(m, rows)),), 255, dtype=torch.uint8, device="cuda")
    got, gb = nf4.nf4_act_backward(mine, pre, "gelu", dz=mine, dbias=bias[:rows], workspace=ws)
    assert got.data_ptr() == room.data_ptr() and torch.equal(mine, dz) and torch.equal(gb, db)
    assert (room[m * rows:] == 7).all() and (bias[rows:] == 7).all()


def test_no_activation_needs_no_pre():
    torch = need_gpu()
    dy = torch.randn((70, 50), device="cuda").bfloat16()
    dz, db = nf4.nf4_act_backward(dy, None, "none")
    assert torch.equal(dz, dy)
    check(torch, "none", dy, None, dz, db)
    with pytest.raises(ValueError):
        nf4.nf4_act_backward(dy, None, "silu")


def test_no_rows():
    torch = need_gpu()
    e = torch.empty((0, 24), dtype=torch.bfloat16, device="cuda")
    dz, db = nf4.nf4_act_backward(e, e, "silu")
    assert tuple(dz.shape) == (0, 24) and tuple(db.shape) == (24,) and (db == 0).all()


def test_offsets_past_32_bits():
    """2^31 elements and more: the last rows, and the sums of ones."""
    torch = need_gpu()
    m, rows = 33000, 65544
    say("act backward", m, rows)
    dy = torch.ones((m, rows), dtype=torch.bfloat16, device="cuda")
    pre = torch.full((m, rows), 3.0, dtype=torch.bfloat16, device="cuda")
    pre[-1] = -2.0
    dz, db = nf4.nf4_act_backward(dy, pre, "relu")
    assert (dz[-1] == 0).all() and (dz[-2] == 1).all() and (dz[16500] == 1).all()
    assert (db == m - 1).all()  # whole numbers below 2^24 add exactly
