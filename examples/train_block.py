"""One residual block trained data-parallel with the library's operators, its
activations kept in 8 bits and its gradients written where the step reads them.

    python examples/train_block.py [--steps K] [--tokens T] [--width D] [--replicas M]

The block is r = x + a * gate * norm(relu(h W1^T) W2^T) with h = w_in * rh(x)
and a final norm; its parameters lie in one flat buffer, as does each of the M
replicas' gradients.  Per replica and step:

 forward   the norm before the block also packs the normalised rows rh into an
           8-bit checkpoint; the hidden activation is packed on its own; the
           norm after the block, its gate and the residual are one call, which
           packs what the backward pass needs.  No bf16 activation is kept.
 backward  the block norms' gradients come from the checkpoints; each weight
           gradient is taken straight from a checkpoint and written into the
           replica's flat gradient buffer.
 step      the fused ZeRO-1 step reads the M buffers, updates the sharded fp32
           state and writes the flat bf16 parameters.

The two plain products (h W1^T, g W2 and so on) are torch's.  The target is a
fixed random map, so the loss falls.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_sharded_mixed_zero1_gb300 as z  # noqa: E402


class Block:
    """Views of one flat bf16 buffer: the parameters, or their gradients."""

    def __init__(self, flat: torch.Tensor, D: int, F: int):
        sizes = self.sizes(D, F)
        parts = torch.split(flat, sizes)
        self.w_in, self.w1, self.w2, self.w_post, self.gate, self.w_out = (
            parts[0], parts[1].view(F, D), parts[2].view(D, F), parts[3], parts[4], parts[5])

    @staticmethod
    def sizes(D: int, F: int) -> list[int]:
        return [D, F * D, D * F, D, D, D]


class Saved:
    """What a replica keeps between its forward and backward pass: 8-bit
    checkpoints and one fp32 statistic per row and norm."""

    def __init__(self, T: int, D: int, F: int, device):
        self.x8, self.y8, self.r8 = (z.new_checkpoint(T, D, device) for _ in range(3))
        self.a8 = z.new_checkpoint(T, F, device)
        self.rstd_in, self.rstd_post, self.rstd_out = (torch.empty(T, device=device) for _ in range(3))

    def nbytes(self) -> int:
        return sum(k.nbytes for k in (self.x8, self.y8, self.r8, self.a8)) + 12 * self.rstd_in.numel()


CFG = z.BlockNorm(eps=1e-6, residual_scale=0.5, gate_act="linear")
NORM = z.BlockNorm(eps=1e-6, residual_scale=0.0)


def forward(p: Block, x: torch.Tensor, s: Saved) -> torch.Tensor:
    """The block's output (the final norm of the residual stream), bf16."""
    h, r, out = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    # the norm before the block: with a residual scale of 0 r is x itself
    z.zero1_block_norm_forward(NORM, x, x, r, h, rstd_pre=s.rstd_in, w_pre=p.w_in, r8=s.x8)
    act = torch.relu(h @ p.w1.t())
    z.zero1_checkpoint_pack(act, s.a8)
    y = act @ p.w2.t()
    z.zero1_block_norm_forward(CFG, y, x, r, out, s.rstd_post, s.rstd_out, w_post=p.w_post, w_pre=p.w_out, gate=p.gate,
                               y8=s.y8, r8=s.r8)
    return out


def backward(p: Block, g: Block, dout: torch.Tensor, s: Saved) -> None:
    """Writes every parameter's gradient into the flat buffer behind g."""
    dx, dy = torch.empty_like(dout), torch.empty_like(dout)
    z.zero1_block_norm_backward(CFG, dout, None, s.y8, s.r8, s.rstd_post, s.rstd_out, dy, dx, w_post=p.w_post,
                                w_pre=p.w_out, gate=p.gate, dw_post=g.w_post, dw_pre=g.w_out, dgate=g.gate)
    z.zero1_weight_grad(dy, s.a8, g.w2)
    act = z.zero1_checkpoint_unpack(s.a8, torch.empty((dy.shape[0], p.w2.shape[1]), dtype=dy.dtype, device=dy.device))
    dact = (dy @ p.w2).mul_(act > 0)
    # h = w_in * rh: the gradient of w1 from the checkpoint of rh, w_in as column scale
    z.zero1_weight_grad(dact, s.x8, g.w1, col_scale=p.w_in)
    dh = dact @ p.w1
    z.zero1_block_norm_backward(NORM, dh, dx, None, s.x8, None, s.rstd_in, dy, torch.empty_like(dx), w_pre=p.w_in,
                                dw_pre=g.w_in)


def train(steps: int = 20, T: int = 512, D: int = 256, M: int = 4, lr: float = 2e-3, device="cuda", seed: int = 0,
          report=None) -> list[float]:
    """Trains from random weights; returns the mean loss of each step."""
    F = 4 * D
    gen = torch.Generator(device=device).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device=device) * std

    n = sum(Block.sizes(D, F))
    plan = z.zero1_plan(n, M, 8, tensor_numels=Block.sizes(D, F))
    master = torch.zeros(plan.padded_n, device=device)
    q = Block(master[:n], D, F)
    for w in (q.w_in, q.w_post, q.w_out, q.gate):
        w.fill_(1.0)
    q.w1.copy_(normal(F, D, std=D ** -0.5))
    q.w2.copy_(normal(D, F, std=F ** -0.5))
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    params = master[:n].to(torch.bfloat16)
    grads = [torch.empty(n, dtype=torch.bfloat16, device=device) for _ in range(M)]
    step = z.FusedStep(plan, 0, M, grads, master, m, v, params)
    p, g = Block(params, D, F), [Block(t, D, F) for t in grads]
    saved = [Saved(T, D, F, device) for _ in range(M)]
    target = normal(D, D, std=D ** -0.5).to(torch.bfloat16)
    xs = [normal(T, D).to(torch.bfloat16) for _ in range(M)]
    goals = [(x @ target).float() for x in xs]
    if report:
        report(f"{n} parameters, {M} replicas of {T} tokens; kept per replica: {saved[0].nbytes()} bytes "
               f"({2 * T * (3 * D + F)} as bf16)")
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
            report(f"step {t}: loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=256)
    ap.add_argument("--replicas", type=int, default=4)
    args = ap.parse_args()
    train(args.steps, args.tokens, args.width, args.replicas, report=print)
