"""The layer calls as a training step uses them: two projections with adapters,
biases and an activation, a router's loss, the backward pass through the frozen
weights, and all gradients clipped together -- against autograd in float64 --
and the same calls on a side stream and in graphs."""

from __future__ import annotations

import math

import pytest

import dequant_matmul_nf4_amd as nf4
from tests.gpu_common import need_gpu, say
from tests.layer_common import act64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _seed():
    need_gpu().manual_seed(47)


def rel(got, want):
    return float((got.double() - want.double()).norm() / want.double().norm())


class Block:
    """h = act(x W1^T + s x A1^T B1^T + b1);  y = h W2^T + s h A2^T B2^T + b2 + x."""

    def __init__(self, torch, hidden=256, wide=640, r=16, act="gelu", experts=8, slots=2):
        def param(*shape, by=1.0):
            return (by * torch.randn(shape, device="cuda"))

        self.torch, self.act, self.s, self.slots, self.experts = torch, act, 2.0, slots, experts
        self.W = [nf4.quantize_weight((param(wide, hidden) / hidden ** 0.5).bfloat16()),
                  nf4.quantize_weight((param(hidden, wide) / wide ** 0.5).bfloat16())]
        self.A = [(param(r, hidden) / hidden ** 0.5).bfloat16(), (param(r, wide) / wide ** 0.5).bfloat16()]
        self.B = [(param(wide, r) * 0.1).bfloat16(), (param(hidden, r) * 0.1).bfloat16()]
        self.b = [param(wide, by=0.3), param(hidden, by=0.3)]
        self.router = (param(experts, hidden) / hidden ** 0.5)

    def step(self, x, dy, most, stream=None):
        """(y, loss, dx, gradients before clipping, clipped, norm)"""
        torch, s = self.torch, self.s
        kw = dict(lora_scale=s, stream=stream)
        h, z = nf4.nf4_linear(self.W[0], x, bias=self.b[0], act=self.act, lora_a=self.A[0], lora_b=self.B[0], save_pre=True, **kw)
        y = nf4.nf4_linear(self.W[1], h, bias=self.b[1], residual=x, lora_a=self.A[1], lora_b=self.B[1], **kw)
        logits = x.float() @ self.router.t()
        ids = logits.topk(self.slots, 1).indices.to(torch.int32).contiguous()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        loss, counts, _ = nf4.nf4_expert_balance(logits, ids, self.slots, 0.1, stream=stream)
        dlogits = nf4.nf4_expert_balance_backward(logits, counts, self.slots, 0.1, stream=stream)
        _, db2 = nf4.nf4_act_backward(dy, None, "none", want=("dbias",), stream=stream)
        dh = nf4.nf4_gemm_dx(self.W[1], dy, lora_a=self.A[1], lora_b=self.B[1], **kw)
        da2, dB2 = nf4.nf4_lora_grads(h, dy, self.A[1], self.B[1], s, stream=stream)
        dz, db1 = nf4.nf4_act_backward(dh, z, self.act, stream=stream)
        dx = nf4.nf4_gemm_dx(self.W[0], dz, lora_a=self.A[0], lora_b=self.B[0], **kw)
        da1, dB1 = nf4.nf4_lora_grads(x, dz, self.A[0], self.B[0], s, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        drouter = dlogits.t() @ x.float()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        grads = [da1, dB1, db1, da2, dB2, db2, drouter]
        out = torch.empty(sum(g.numel() for g in grads), device="cuda")
        if stream is not None:
            out.record_stream(stream)
            drouter.record_stream(stream)
        norm, _ = nf4.nf4_grad_clip(grads, most, out=out, stream=stream)
        return y, loss, dx, grads, out, norm

    def reference(self, x, dy):
        """Autograd in float64 over the dequantized weights."""
        torch = self.torch
        leaves = [t.double().requires_grad_(True) for pair in zip(self.A, self.B, self.b) for t in pair]
        a1, b1, c1, a2, b2, c2 = leaves
        router, xd = self.router.double().requires_grad_(True), x.double().requires_grad_(True)
        w1, w2 = (nf4.nf4_dequantize(w, out_dtype=torch.bfloat16).double() for w in self.W)
        h = act64(torch, self.act, xd @ w1.t() + self.s * (xd @ a1.t()) @ b1.t() + c1)
        y = h @ w2.t() + self.s * (h @ a2.t()) @ b2.t() + c2 + xd
        xr = x.double()
        logits = xr @ router.t()
        ids = (x.float() @ self.router.t()).topk(self.slots, 1).indices
        c = torch.bincount(ids.reshape(-1), minlength=self.experts).double()
        t = x.shape[0]
        loss = 0.1 * self.experts * (c / (t * self.slots) * torch.softmax(logits, 1).mean(0)).sum()
        grads = torch.autograd.grad((y * dy.double()).sum() + loss, leaves + [router, xd])
        order = [grads[0], grads[1], grads[2], grads[3], grads[4], grads[5], grads[6]]
        return y, loss, grads[7] - dy.double(), order


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("m", [24, 300])
def test_step_against_autograd(act, m):
    """Relative Frobenius errors: each bf16 rounding on the way (h, z, dh, dz, the weights of
    each product) adds at most 2^-8 / sqrt(3) = 2.3e-3 in the mean square; six of them, 6e-3.
    relu's slope flips where z's error d crosses zero: with z normal of deviation 1 a share of
    0.4 E|d| of the values, E|d| at most sqrt(2) 2.3e-3 sqrt(2 / pi) = 2.6e-3 (the weights' and x's
    roundings on both sides), so 1e-3 of them; each is wrong by its whole gradient, and half of all
    have one: sqrt(2 1e-3) = 4.6e-2 of what passes the activation."""
    torch = need_gpu()
    say("layer step", act, m)
    block = Block(torch, act=act)
    x, dy = torch.randn((m, 256), device="cuda").bfloat16(), torch.randn((m, 256), device="cuda").bfloat16()
    y, loss, dx, grads, out, norm = block.step(x, dy, 1.0)
    ry, rl, rdx, rgrads = block.reference(x, dy)
    past = 5e-2 if act == "relu" else 1e-2  # what passes the activation's slope
    assert rel(y, ry.detach()) < 1e-2 and rel(dx, rdx) < past
    assert abs(float(loss) - float(rl.detach())) < 1e-5 * float(rl.detach())
    for i, (g, r) in enumerate(zip(grads, rgrads)):
        assert rel(g.reshape(r.shape), r) < (past if i < 3 else 1e-2 if i < 6 else 1e-4), i
    n = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(norm) - n) < 1e-6 * n
    flat = torch.cat([g.reshape(-1) for g in grads]).double()
    assert rel(out, flat / (n + 1e-6)) < 1e-6


def test_side_stream():
    """On a side stream, the binding's buffers kept until it is through."""
    torch = need_gpu()
    block = Block(torch)
    x, dy = torch.randn((90, 256), device="cuda").bfloat16(), torch.randn((90, 256), device="cuda").bfloat16()
    ref = block.step(x, dy, 0.5)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = block.step(x, dy, 0.5, stream=side)
    junk = [torch.full((t.numel() * t.element_size(),), 0xA5, dtype=torch.uint8, device="cuda") for t in got[3] for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    del junk
    for a, b in zip(list(ref[:3]) + ref[3] + list(ref[4:]), list(got[:3]) + got[3] + list(got[4:])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("m", [1, 12, 48, 300])
def test_graphs(m):
    """Two graphs of the calls, which share a workspace and are replayed in turn with other
    inputs and eager work between: each replay equals the eager calls bit for bit."""
    torch = need_gpu()
    say("layer graphs", m)
    rows, cols, r, experts = 264, 320, 8, 16
    W = nf4.quantize_weight((torch.randn((rows, cols), device="cuda") / 18).bfloat16())
    A = (torch.randn((r, cols), device="cuda") / 18).bfloat16()
    B = torch.randn((rows, r), device="cuda").bfloat16()
    bias = torch.randn(rows, device="cuda")
    tokens = 40 * m
    names = max(nf4.nf4_linear_workspace(m, rows, cols, r), nf4.nf4_act_backward_workspace(m, rows),
                nf4.nf4_expert_balance_workspace(tokens, experts), nf4.nf4_grad_workspace(300))
    ws = torch.empty(names, dtype=torch.uint8, device="cuda")

    def inputs():
        return dict(x=torch.randn((m, cols), device="cuda").bfloat16(), dy=torch.randn((m, rows), device="cuda").bfloat16(),
                    logits=torch.randn((tokens, experts), device="cuda"), dloss=torch.rand(1, device="cuda"),
                    ids=torch.randint(-1, experts, (tokens, 2), dtype=torch.int32, device="cuda"),
                    grads=[torch.randn(900 + i, device="cuda") for i in range(300)])

    def outputs():
        new = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
        f = torch.float32
        return dict(y=new(m, rows), pre=new(m, rows), dz=new(m, rows), db=new(rows, dtype=f), loss=new(1, dtype=f),
                    counts=new(experts + 1, dtype=torch.int32), mean=new(experts, dtype=f), dlogits=new(tokens, experts, dtype=f),
                    norm=new(1, dtype=f), out=new(sum(900 + i for i in range(300)), dtype=f), n2=new(1, dtype=f))

    def path(i, o):
        nf4.nf4_linear(W, i["x"], bias=bias, act="gelu", residual=i["dy"], lora_a=A, lora_b=B, lora_scale=2.0, y=o["y"], pre=o["pre"],
                       workspace=ws)
        nf4.nf4_act_backward(i["dy"], o["pre"], "gelu", dz=o["dz"], dbias=o["db"], workspace=ws)
        nf4.nf4_expert_balance(i["logits"], i["ids"], 2, 0.1, loss=o["loss"], counts=o["counts"], mean_probs=o["mean"], workspace=ws)
        nf4.nf4_expert_balance_backward(i["logits"], o["counts"], 2, 0.1, dloss=i["dloss"], dlogits=o["dlogits"])
        nf4.nf4_grad_clip(i["grads"], 3.0, out=o["out"], norm=o["norm"], workspace=ws)
        nf4.nf4_grad_norm(i["grads"][:50], norm=o["n2"], workspace=ws)

    sets = [(inputs(), outputs()) for _ in range(2)]
    for i, o in sets:
        path(i, o)
    torch.cuda.synchronize()
    graphs = []
    for i, o in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="relaxed"):
            path(i, o)
        graphs.append(g)
    for rep in range(3):
        for (i, o), g in zip(sets, graphs):
            fresh = inputs()
            for k, v in fresh.items():
                for a, b in zip(i[k] if k == "grads" else [i[k]], v if k == "grads" else [v]):
                    a.copy_(b)
            want = outputs()
            path(i, want)
            for v in o.values():
                v.zero_()
            ws.fill_(255)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for k in o:
                assert torch.equal(o[k], want[k]), (rep, k)
