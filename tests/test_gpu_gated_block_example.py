"""Layer norm, gated feed-forward block, weight gradients, clipping and step
together, as examples/train_gated_block.py uses them: gradients against automatic
differentiation in float64, one step against its formula, and training."""
import importlib.util
import math
import os

import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_gated_block", os.path.join(ROOT, "examples", "train_gated_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm(t):
    d = t - t.mean(1, keepdim=True)
    return d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt()


def setup(example, T, D, F, offset):
    g = torch.Generator().manual_seed(3)
    n = sum(example.Block.sizes(D, F))
    flat = torch.zeros(n + offset, dtype=torch.bfloat16)
    p = example.Block(flat[offset:], D, F)
    for w in (p.ln_w, p.out_w):
        w.copy_(1 + 0.2 * torch.randn(D, generator=g))
    for w in (p.ln_b, p.out_b):
        w.copy_(0.2 * torch.randn(D, generator=g))
    for w, fan in ((p.w_gate, D), (p.w_up, D), (p.w_down, F)):
        w.copy_(torch.randn(w.shape, generator=g) * fan ** -0.5)
    x = (torch.randn((T, D), generator=g) + 0.3).to(torch.bfloat16)
    dout = (torch.randn((T, D), generator=g) * 1e-2).to(torch.bfloat16)
    return n, flat, x, dout


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,D,F,offset", [(96, 136, 360, 3), (200, 128, 384, 0), (33, 77, 150, 1)])
def test_gradients_against_autograd(cuda_device, example, T, D, F, offset, act):
    n, flat, x, dout = setup(example, T, D, F, offset)
    q = flat.double()[offset:].clone().requires_grad_()
    b = example.Block(q, D, F)
    xd = x.double().requires_grad_()
    h = norm(xd) * b.ln_w + b.ln_b
    g = h @ b.w_gate.t()
    f = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    out = norm(xd + 0.5 * ((f * (h @ b.w_up.t())) @ b.w_down.t())) * b.out_w + b.out_b
    out.backward(dout.double())

    gpu = flat.to(cuda_device)
    grads = torch.zeros(n + offset, dtype=torch.bfloat16, device=cuda_device)
    s = example.Saved(T, D, cuda_device)
    pg = example.Block(gpu[offset:], D, F)
    got = example.forward(pg, x.to(cuda_device), s, act)
    dx = example.backward(pg, example.Block(grads[offset:], D, F), dout.to(cuda_device), s, act)
    assert (got.cpu().double() - out.detach()).norm() <= 0.02 * out.norm()  # five bf16 tensors on the way, 2^-8 each at most
    # the checkpoints' e4m3 codes are within 2^-4 of their values, 0.026 in the mean square
    assert (dx.cpu().double() - xd.grad).norm() <= 0.08 * xd.grad.norm()
    want, have = example.Block(q.grad, D, F), example.Block(grads[offset:].double().cpu(), D, F)
    for name in example.NAMES:
        a, c = getattr(want, name), getattr(have, name)
        assert (a - c).norm() <= 0.08 * a.norm(), name
    assert (grads[:offset] == 0).all()


@pytest.mark.parametrize("max_norm", [1e-4, 1e3])
def test_one_step(cuda_device, example, max_norm):
    """Replicas' gradients from the block, then norm, clipping and AdamW against
    their formulas in float64."""
    T, D, F, M = 64, 64, 136, 3
    n, flat, x, dout = setup(example, T, D, F, 0)
    params = flat.to(cuda_device)
    plan = z.zero1_plan(n, M, 8)
    master = torch.zeros(plan.padded_n, device=cuda_device)
    master[:n] = params.float()
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    grads = [torch.empty(n, dtype=torch.bfloat16, device=cuda_device) for _ in range(M)]
    s = example.Saved(T, D, cuda_device)
    for r in range(M):
        example.forward(example.Block(params, D, F), x.roll(r, 0).to(cuda_device), s)
        example.backward(example.Block(params, D, F), example.Block(grads[r], D, F), (dout * (r + 1)).to(cuda_device), s)
    start = master.double()
    step = example.ClippedStep(plan, grads, master, m, v, params, max_norm)
    hp = z.AdamW(lr=1e-3, weight_decay=0.1, global_batch=M * T, step=1)
    step(hp)
    g = sum(t.double() for t in grads) / (M * T)
    norm64 = g.norm().item()
    assert abs(step.norm.item() - norm64) <= 1e-5 * norm64 and step.flag.item() == 0
    assert (norm64 > max_norm) == (max_norm < 1)  # one of the two is clipped
    g = g * min(1.0, max_norm / (norm64 + 1e-6))
    w = start[:n] * (1 - 1e-4)
    w -= 1e-3 * g / (g.abs() + 1e-8)  # the first step: m / (1 - beta1) over the root of v / (1 - beta2)
    # where |g| is near eps the quotient moves with g's own rounding, a few 2^-24 of it
    assert (master[:n].double() - w).abs().max().item() <= 1e-3 * 2e-6 + 2.0 ** -23 * w.abs().max().item()
    assert torch.equal(params, master[:n].to(torch.bfloat16))
    assert math.isfinite(norm64)


def test_training_runs(cuda_device, example):
    losses = example.train(steps=4, T=130, D=96, F=264, M=2, device=cuda_device)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)
    assert z.zero1_device_status() == 0
