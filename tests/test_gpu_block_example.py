"""The operators together, as examples/train_block.py uses them: gradients in
the replicas' flat buffers against automatic differentiation, and training."""
import importlib.util
import os

import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_against_autograd(cuda_device, example):
    T, D = 96, 136                                    # rows that end inside a stage, a width of no power of two
    F, dev = 4 * D, cuda_device
    g = torch.Generator().manual_seed(3)
    n = sum(example.Block.sizes(D, F))
    flat = torch.zeros(n + 3, dtype=torch.bfloat16)   # an odd element offset, as inside a larger flat buffer
    p = example.Block(flat[3:], D, F)
    for w in (p.w_in, p.w_post, p.w_out, p.gate):
        w.copy_(1 + 0.2 * torch.randn(D, generator=g))
    p.w1.copy_(torch.randn((F, D), generator=g) * D ** -0.5)
    p.w2.copy_(torch.randn((D, F), generator=g) * F ** -0.5)
    x = torch.randn((T, D), generator=g).to(torch.bfloat16)
    dout = (torch.randn((T, D), generator=g) * 1e-2).to(torch.bfloat16)

    q = flat.double()[3:].clone().requires_grad_()
    b = example.Block(q, D, F)
    xd = x.double()
    rms = lambda t: t * (t.square().mean(1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    y = torch.relu((rms(xd) * b.w_in) @ b.w1.t()) @ b.w2.t()
    out = rms(xd + 0.5 * b.gate * (rms(y) * b.w_post)) * b.w_out
    out.backward(dout.double())

    gpu = flat.to(dev)
    grads = torch.zeros(n + 3, dtype=torch.bfloat16, device=dev)
    s = example.Saved(T, D, F, dev)
    pg = example.Block(gpu[3:], D, F)
    got = example.forward(pg, x.to(dev), s)
    example.backward(pg, example.Block(grads[3:], D, F), dout.to(dev), s)
    assert (got.cpu().double() - out.detach()).norm() <= 0.01 * out.norm()   # a few bf16 roundings of 2^-9
    want, have = example.Block(q.grad, D, F), example.Block(grads[3:].double().cpu(), D, F)
    for name in ("w_in", "w1", "w2", "w_post", "gate", "w_out"):
        a, c = getattr(want, name), getattr(have, name)
        # an e4m3 code is within 2^-4 of its value, 0.026 in the mean square; the
        # codes of three tensors and the relu's edge enter each gradient
        assert (a - c).norm() <= 0.08 * a.norm(), name
    assert (grads[:3] == 0).all()


def test_training_lowers_the_loss(cuda_device, example):
    """Full-batch training on a fixed target: the last loss is the lowest."""
    losses = example.train(steps=12, T=200, D=128, M=3, device=cuda_device)
    assert losses[-1] == min(losses) < losses[0]
    assert z.zero1_device_status() == 0
