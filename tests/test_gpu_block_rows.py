"""Block norms with many rows per block: a row's results are those of the row
alone, whatever its block did before."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


class Rows:
    """Inputs on the GPU whose statistics differ from row to row."""

    def __init__(self, T, D, act, res, post, pre, gate, cuda, gate_act="linear", ckpt=False):
        g = torch.Generator(device=cuda).manual_seed(T + D)
        spread = torch.exp(torch.randn((T, 1), generator=g, device=cuda))
        r = lambda *s: torch.randn(s, generator=g, device=cuda)  # noqa: E731
        self.T, self.D, self.ckpt = T, D, ckpt
        self.y, self.x = (r(T, D) * spread).to(act), (r(T, D) * spread.flip(0)).to(res)
        self.w_post = (1 + 0.1 * r(D)).to(BF16) if post else None
        self.w_pre = (1 + 0.1 * r(D)).to(BF16) if pre else None
        shape = {None: None, "channel": (D,), "token": (T, 1), "full": (T, D)}[gate]
        self.gate = None if shape is None else (0.5 + 0.5 * r(*shape)).to(BF16)
        # gradients along the rows themselves: means that differ and matter
        self.dh = (spread * (r(T, D) + self.x.float() / spread.flip(0))).to(act) if pre else None
        self.dr = (spread * (r(T, D) + self.y.float() / spread)).to(res)
        self.cfg = z.BlockNorm(residual_scale=0.7, gate_act=gate_act)

    def part(self, a, b):
        """The calls on rows [a, b): every per-row output, in order."""
        cut = lambda t: None if t is None else t[a:b]  # noqa: E731
        per_row = self.gate is not None and self.gate.dim() == 2
        gate = cut(self.gate) if per_row else self.gate
        y, x, n, dev = self.y[a:b], self.x[a:b], b - a, self.y.device
        r, dx, dy = torch.empty_like(x), torch.empty_like(x), torch.empty_like(y)
        h = torch.empty_like(y) if self.w_pre is not None else None
        rstd_post = torch.empty(n, device=dev) if self.w_post is not None else None
        rstd_pre = torch.empty(n, device=dev) if self.w_pre is not None else None
        y8 = z.new_checkpoint(n, self.D, dev) if self.ckpt else None
        r8 = z.new_checkpoint(n, self.D, dev) if self.ckpt and self.w_pre is not None else None
        w = dict(w_post=self.w_post, w_pre=self.w_pre, gate=gate)
        z.zero1_block_norm_forward(self.cfg, y, x, r, h, rstd_post, rstd_pre, y8=y8, r8=r8, **w)
        need_y = self.w_post is not None or gate is not None
        dgate = torch.empty_like(gate) if per_row else None
        z.zero1_block_norm_backward(self.cfg, cut(self.dh), self.dr[a:b], (y8 if self.ckpt else y) if need_y else None,
                                    None if self.w_pre is None else r8 if self.ckpt else r, rstd_post, rstd_pre, dy, dx,
                                    dgate=dgate, **w)
        out = [r, h, rstd_post, rstd_pre, dx, dy, dgate]
        if self.ckpt:
            out += [y8.codes, y8.exps[:, :n].t()] + ([r8.codes, r8.exps[:, :n].t()] if r8 is not None else [])
        return [t.clone() for t in out if t is not None]


def check_rows_alone(p, at_once):
    """All rows in one call against `at_once` rows at a time, bit for bit: a
    row's arithmetic does not depend on its block."""
    whole = p.part(0, p.T)
    for a in range(0, p.T, at_once):
        b = min(p.T, a + at_once)
        for k, (got, want) in enumerate(zip(whole, p.part(a, b))):
            assert torch.equal(got[a:b], want), (k, a)
    assert all(torch.isfinite(t.float()).all() for t in whole if t.dtype is not torch.uint8)


@pytest.mark.parametrize("T,D,act,res", [
    (2000, 9000, BF16, BF16), (1500, 16384, BF16, BF16), (1200, 8193, F32, F32),   # above the ring's widths
    (3000, 1600, BF16, BF16), (2000, 8192, BF16, F32), (2500, 2000, F32, F32)])    # rows that may not fit the ring
@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (True, True), (False, False)])
@pytest.mark.parametrize("gate", [None, "channel"])
def test_a_row_does_not_depend_on_its_block(cuda_device, T, D, act, res, post, pre, gate):
    check_rows_alone(Rows(T, D, act, res, post, pre, gate, cuda_device), 150)
