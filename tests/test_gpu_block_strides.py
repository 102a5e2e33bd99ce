"""Inputs whose rows repeat (a stride of 0) or overlap (a stride below the
width): the same results, bit for bit, as from rows that lie apart, at the same
place modulo 16 bytes (above 8192 columns the order of a row's sum depends on
whether its rows are aligned)."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rows(T, D, ld, dtype, cuda, seed, off=0):
    """A [T, D] view with rows `ld` apart of random values."""
    g = torch.Generator(device=cuda).manual_seed(seed)
    flat = torch.randn(off + (T - 1) * ld + D, generator=g, device=cuda).to(dtype)
    return flat.as_strided((T, D), (ld, 1), off)


def apart(t):
    """A copy of such a view whose rows do not share an element."""
    (T, D), ld, off = t.shape, t.stride(0), t.storage_offset()
    wide = -(-D // 8) * 8 + ld % 8
    flat = torch.zeros(off + T * wide, dtype=t.dtype, device=t.device)
    v = flat.as_strided((T, D), (wide, 1), off)
    v.copy_(t)
    return v


STRIDES = [(300, 1024, 0, 0), (300, 1024, 8, 0), (300, 1024, 1, 0), (300, 1021, 0, 1), (300, 1021, 7, 1), (40, 9000, 0, 0),
           (40, 9000, 4, 3), (300, 200, 64, 0)]


@pytest.mark.parametrize("T,D,ld,off", STRIDES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pack(cuda_device, T, D, ld, off, dtype):
    x = rows(T, D, ld, dtype, cuda_device, 1, off)
    a, b = z.new_checkpoint(T, D, cuda_device), z.new_checkpoint(T, D, cuda_device)
    z.zero1_checkpoint_pack(x, a)
    z.zero1_checkpoint_pack(apart(x), b)
    assert torch.equal(a.codes, b.codes) and torch.equal(a.exps[:, :T], b.exps[:, :T])


@pytest.mark.parametrize("T,D,ld,off", STRIDES)
@pytest.mark.parametrize("act,res", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("gate", ["full", "token"])
def test_block_norms(cuda_device, T, D, ld, off, act, res, gate):
    y, x = rows(T, D, ld, act, cuda_device, 2, off), rows(T, D, ld, res, cuda_device, 3, off)
    dh, dr = rows(T, D, ld, act, cuda_device, 4, off), rows(T, D, ld, res, cuda_device, 5, off)
    gt = rows(T, D, ld, BF16, cuda_device, 6, off) if gate == "full" else rows(T, 1, ld, BF16, cuda_device, 6, off)
    w = torch.rand(D, device=cuda_device).to(BF16) + 1
    cfg = z.BlockNorm(residual_scale=0.5, gate_act="sigmoid")
    got = []
    for c in (lambda t: t, apart):
        r, h = torch.empty((T, D), dtype=res, device=cuda_device), torch.empty((T, D), dtype=act, device=cuda_device)
        a, b = torch.empty(T, device=cuda_device), torch.empty(T, device=cuda_device)
        z.zero1_block_norm_forward(cfg, c(y), c(x), r, h, a, b, w_post=w, w_pre=w, gate=c(gt))
        dx, dy = torch.empty_like(r), torch.empty_like(h)
        dw1, dw2 = torch.empty(D, device=cuda_device), torch.empty(D, device=cuda_device)
        dg = torch.empty(gt.shape, dtype=BF16 if gate == "full" else F32, device=cuda_device)
        z.zero1_block_norm_backward(cfg, c(dh), c(dr), c(y), c(x), a, b, dy, dx, w_post=w, w_pre=w, gate=c(gt), dw_post=dw1,
                                    dw_pre=dw2, dgate=dg)
        got.append((r, h, a, b, dx, dy, dw1, dw2, dg))
    for k, (p, q) in enumerate(zip(*got)):
        assert torch.equal(p, q), k


@pytest.mark.parametrize("T,N,ld,off", [(300, 512, 0, 0), (300, 512, 8, 0), (300, 512, 64, 8), (300, 512, 3, 0), (300, 511, 0, 1),
                                        (2000, 264, 16, 0), (1, 264, 0, 0)])
@pytest.mark.parametrize("out", [BF16, F32])
def test_weight_grad(cuda_device, T, N, ld, off, out):
    dy = rows(T, N, ld, BF16, cuda_device, 7, off)
    k = z.new_checkpoint(T, 200, cuda_device)
    z.zero1_checkpoint_pack(rows(T, 200, 200, F32, cuda_device, 8), k)
    a, b = (torch.empty((N, 200), dtype=out, device=cuda_device) for _ in range(2))
    z.zero1_weight_grad(dy, k, a)
    z.zero1_weight_grad(apart(dy), k, b)
    assert torch.equal(a, b)
