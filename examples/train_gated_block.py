"""One pre-norm block with a layer norm and a gated feed-forward part, trained
data-parallel: gradients in the replicas' flat buffers, clipped to a global norm
inside the optimizer step.

    python examples/train_gated_block.py [--steps K] [--tokens T] [--width D] [--inner F] [--replicas M]

The block is r = x + a * (act(h Wg^T) * (h Wu^T)) Wd^T with h = ln(x), and out =
ln(r).  Per replica and step:

 forward   layer norm, the gated feed-forward block in one kernel, the down
           projection, then residual and last norm in one call.  Kept: the first
           norm's rows as an 8-bit checkpoint and h; neither g, u nor the
           feed-forward activation.
 backward  the last norm's gradients, the down projection's, and then the
           feed-forward block's with its pre-activations computed again, which
           also gives the activation that the down projection's weight gradient
           takes.  Each weight gradient is written into the replica's flat buffer.
 step      the sum of squares of the replicas' summed gradients, shard by shard as
           ranks would, then the fused step with those gradients clipped.

The two plain products (a Wd^T and dy Wd) are torch's.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_zero1_gb300 as z  # noqa: E402

NAMES = ("ln_w", "ln_b", "w_gate", "w_up", "w_down", "out_w", "out_b")
IN, OUT = z.LayerNorm(eps=1e-5), z.LayerNorm(eps=1e-5, residual_scale=0.5)


class Block:
    """Views of one flat buffer: the parameters, or their gradients."""

    def __init__(self, flat: torch.Tensor, D: int, F: int):
        shapes = [(D,), (D,), (F, D), (F, D), (D, F), (D,), (D,)]
        for name, part, shape in zip(NAMES, torch.split(flat, self.sizes(D, F)), shapes):
            setattr(self, name, part.view(shape))

    @staticmethod
    def sizes(D: int, F: int) -> list[int]:
        return [D, D, F * D, F * D, D * F, D, D]


class Saved:
    """What a replica keeps between its forward and backward pass."""

    def __init__(self, T: int, D: int, device):
        self.h = torch.empty((T, D), dtype=torch.bfloat16, device=device)
        self.x8, self.r8 = z.new_checkpoint(T, D, device), z.new_checkpoint(T, D, device)
        self.mean, self.rstd, self.out_mean, self.out_rstd = (torch.empty(T, device=device) for _ in range(4))


def forward(p: Block, x: torch.Tensor, s: Saved, act: str = "silu") -> torch.Tensor:
    """The block's output, bf16 [T, D]."""
    T, F = x.shape[0], p.w_gate.shape[0]
    z.zero1_layer_norm_forward(IN, x, s.h, s.mean, s.rstd, w=p.ln_w, b=p.ln_b, r8=s.x8)
    a = torch.empty((T, F), dtype=x.dtype, device=x.device)
    z.zero1_gated_ffn_forward(s.h, p.w_gate, p.w_up, a, act=act)
    y = a @ p.w_down.t()
    out, r = torch.empty_like(x), torch.empty_like(x)
    z.zero1_layer_norm_forward(OUT, x, out, s.out_mean, s.out_rstd, w=p.out_w, b=p.out_b, y=y, r=r, r8=s.r8)
    return out


def backward(p: Block, g: Block, dout: torch.Tensor, s: Saved, act: str = "silu") -> torch.Tensor:
    """Writes every parameter's gradient into the flat buffer behind g; returns
    the gradient of x."""
    dr, dy = torch.empty_like(dout), torch.empty_like(dout)
    z.zero1_layer_norm_backward(OUT, dout, None, s.r8, s.out_mean, s.out_rstd, dr, dy=dy, w=p.out_w, dw=g.out_w, db=g.out_b)
    da = dy @ p.w_down
    a, du = torch.empty_like(da), torch.empty_like(da)
    dg = da  # in the place of da
    z.zero1_gated_ffn_backward(da, s.h, p.w_gate, p.w_up, dg, du, a=a, act=act)
    z.zero1_weight_grad_bf16(dy, a, g.w_down)
    z.zero1_weight_grad_bf16(dg, s.h, g.w_gate)
    z.zero1_weight_grad_bf16(du, s.h, g.w_up)
    dh, dx = torch.empty_like(dout), torch.empty_like(dout)
    z.zero1_gated_ffn_input_grad(dg, du, p.w_gate, p.w_up, dh)
    z.zero1_layer_norm_backward(IN, dh, dr, s.x8, s.mean, s.rstd, dx, w=p.ln_w, dw=g.ln_w, db=g.ln_b)
    return dx


class ClippedStep:
    """The step over all shards with one global norm, each shard's part of it
    taken on its own as ranks would."""

    def __init__(self, plan, grads, master, m, v, params, max_norm: float):
        self.plan, self.grads, self.state, self.params, self.max_norm = plan, grads, (master, m, v), params, max_norm
        self.sumsq = torch.zeros(1, dtype=torch.float64, device=master.device)
        self.norm = torch.zeros(1, device=master.device)
        self.flag = torch.zeros(1, dtype=torch.int32, device=master.device)

    def __call__(self, hp) -> None:
        M = self.plan.M
        for k in range(M):
            base, _, nv = self.plan.shard_range(k, k + 1)
            z.zero1_shard_grad_sumsq(self.plan, k, k + 1, [g[base:base + nv] for g in self.grads], hp, self.sumsq,
                                     accumulate=k > 0)
        z.zero1_step_clipped(self.plan, 0, M, self.grads, *self.state, self.params, hp, self.sumsq, self.max_norm,
                             norm=self.norm, overflow_flag=self.flag)


def train(steps: int = 20, T: int = 512, D: int = 256, F: int = 704, M: int = 4, lr: float = 2e-3, max_norm: float = 0.5,
          device="cuda", seed: int = 0, report=None) -> list[float]:
    """Trains from random weights; returns the mean loss of each step."""
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=device) * std

    sizes = Block.sizes(D, F)
    n = sum(sizes)
    plan = z.zero1_plan(n, M, 8, tensor_numels=sizes)
    master = torch.zeros(plan.padded_n, device=device)
    q = Block(master[:n], D, F)
    q.ln_w.fill_(1.0)
    q.out_w.fill_(1.0)
    for w, fan in ((q.w_gate, D), (q.w_up, D), (q.w_down, F)):
        w.copy_(normal(*w.shape, std=fan ** -0.5))
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    params = master[:n].to(torch.bfloat16)
    grads = [torch.empty(n, dtype=torch.bfloat16, device=device) for _ in range(M)]
    step = ClippedStep(plan, grads, master, m, v, params, max_norm)
    p, g = Block(params, D, F), [Block(t, D, F) for t in grads]
    saved = [Saved(T, D, device) for _ in range(M)]
    target = normal(D, D, std=D ** -0.5).to(torch.bfloat16)
    xs = [normal(T, D).to(torch.bfloat16) for _ in range(M)]
    goals = [(x @ target).float() for x in xs]
    losses = []
    for t in range(1, steps + 1):
        total = torch.zeros((), device=device)
        for r in range(M):
            diff = forward(p, xs[r], saved[r]).float() - goals[r]
            total += diff.square().mean() / M
            # the sum over this replica's samples; the step divides by the global batch M T
            backward(p, g[r], (diff * (2.0 / D)).to(torch.bfloat16), saved[r])
        step(z.AdamW(lr=lr, beta1=0.9, beta2=0.95, weight_decay=0.0, global_batch=M * T, step=t))
        losses.append(total.item())
        if report and (t == 1 or t % 5 == 0):
            report(f"step {t}: loss {losses[-1]:.4f}, gradient norm {step.norm.item():.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--inner", type=int, default=704)
    ap.add_argument("--replicas", type=int, default=4)
    args = ap.parse_args()
    train(args.steps, args.tokens, args.width, args.inner, args.replicas, report=print)
