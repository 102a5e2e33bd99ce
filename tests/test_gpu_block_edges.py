"""The block norms at the edges of their buffers: what lies behind a vector or
between a matrix's rows reaches no result."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
from zero_sharded_mixed_zero1_gb300 import block as zb
import block_reference as ref
import test_gpu_block_ops as ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def among_nans(t, cuda, pad=0, off=0):
    """ops.dev with NaN in place of every element around t: 16 behind it, `off`
    before it, `pad` after each row."""
    if t is None:
        return None
    rows, D = (1, t.shape[0]) if t.dim() == 1 else t.shape
    pad = 0 if t.dim() == 1 else pad
    big = torch.full((off + rows * (D + pad) + 16,), float("nan"), dtype=t.dtype, device=cuda)
    v = big[off:off + rows * (D + pad)].view(rows, D + pad)[:, :D]
    v.copy_(t.view(rows, D))
    return v[0] if t.dim() == 1 else v


@pytest.fixture
def surrounded(monkeypatch):
    monkeypatch.setattr(ops, "dev", among_nans)


@pytest.mark.parametrize("T,D", [(3, 1), (3, 7), (5, 250), (2, 513), (4, 1021), (3, 2003), (2, 4093), (2, 8190), (2, 9001)])
@pytest.mark.parametrize("act,res", ops.TYPES)
@pytest.mark.parametrize("gate", [None, "channel", "full"])
@pytest.mark.parametrize("param", [BF16, F32])
def test_nothing_behind_a_vector_is_read(cuda_device, surrounded, T, D, act, res, gate, param):
    p = ops.Problem(T, D, act, res, True, True, gate, "sigmoid" if T % 2 else "linear", param=param, seed=20)
    ops.check_forward(p, ops.run_forward(p, cuda_device))
    for ckpt in (False, True):
        ops.check_backward(p, *ops.run_backward(p, cuda_device, ckpt))


@pytest.mark.parametrize("post,pre", [(True, False), (False, True)])
def test_nothing_behind_a_vector_is_read_with_a_norm_left_out(cuda_device, surrounded, post, pre):
    for D in (250, 1021, 2003):
        p = ops.Problem(4, D, BF16, BF16, post, pre, "channel", "linear", seed=21)
        ops.check_forward(p, ops.run_forward(p, cuda_device))
        for ckpt in (False, True):
            ops.check_backward(p, *ops.run_backward(p, cuda_device, ckpt))


@pytest.mark.parametrize("pad,off", [(8, 0), (8, 8), (3, 1), (5, 0), (0, 3)])
@pytest.mark.parametrize("D", [1024, 1021])
def test_nothing_between_rows_is_read(cuda_device, surrounded, pad, off, D):
    for gate in ("channel", "token", "full"):
        p = ops.Problem(9, D, BF16, F32, True, True, gate, "sigmoid", seed=22)
        ops.check_forward(p, ops.run_forward(p, cuda_device, pad, off, woff=off))
        ops.check_backward(p, *ops.run_backward(p, cuda_device, False, pad, off, goff=off))


@pytest.mark.parametrize("D", [640, 1021, 9000])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_a_saved_block_output_that_is_not_needed_is_not_read(cuda_device, D, gate):
    """Without the norm after the block, y serves dgate only: a checkpoint that
    is no use (codes at an odd address, scales that stand for NaN) changes
    nothing, and neither does a tensor over the outputs."""
    p = ops.Problem(40, D, BF16, BF16, False, True, gate, "sigmoid", seed=23)
    T, dev = p.T, cuda_device
    f = p.forward64()
    r, rstd = f["r"].to(BF16).to(dev), f["rstd_pre"].float().to(dev)
    w, g, dh, dr = p.w_pre.to(dev), None if gate is None else p.gate.to(dev), p.dh.to(dev), p.dr.to(dev)
    wide = ref.up(D)
    odd = torch.zeros(T * wide + 1, dtype=torch.uint8, device=dev)[1:].view(T, wide)
    useless = z.Checkpoint8(T, D, odd, torch.full((wide // 128, 128), 255, dtype=torch.uint8, device=dev))
    results = []
    for y in (None, useless, "dy"):
        dy, dx, dw = torch.empty_like(dh), torch.empty_like(dr), torch.empty(D, device=dev)
        z.zero1_block_norm_backward(p.cfg, dh, dr, dy if isinstance(y, str) else y, r, None, rstd, dy, dx, w_pre=w, gate=g,
                                    dw_pre=dw)
        results.append((dy, dx, dw))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    assert all(torch.isfinite(t.float()).all() for t in results[0])


@pytest.mark.parametrize("value", [1.0, float("nan"), float("inf")])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_sums_over_no_rows_do_not_look_at_the_gate(cuda_device, value, kind):
    """Sums over no rows are +0, or stay, whatever a sigmoid gate holds, and at
    an address that its type does not allow."""
    D = 200
    w = torch.ones(D, dtype=BF16, device=cuda_device)
    gate = torch.full((D,), value, dtype=kind, device=cuda_device)
    e, s = torch.empty((0, D), dtype=BF16, device=cuda_device), torch.empty(0, device=cuda_device)
    cfg = z.BlockNorm(gate_act="sigmoid")
    for accumulate, want in ((False, 0.0), (True, 3.0)):
        dw = [torch.full((D,), 3.0, dtype=F32, device=cuda_device) for _ in range(3)]
        z.zero1_block_norm_backward(cfg, e, e, e, e, s, s, e, e, w_post=w, w_pre=w, gate=gate, dw_post=dw[0], dw_pre=dw[1],
                                    dgate=dw[2], accumulate=accumulate)
        assert all((t == want).all() for t in dw)
        if not accumulate:
            assert all(not torch.signbit(t).any() for t in dw)
    dgate = torch.full((D,), 3.0, dtype=F32, device=cuda_device)
    c = zb._CFG.pack(0, D, 1e-6, 1.0, 0, 0, 0, 1, 1, 1, 1, 0)   # fp32 gate and gradients, per channel, sigmoid
    odd = torch.full((D + 1,), value, dtype=F32, device=cuda_device)
    io = zb._BWD.pack(*([0] * 6), odd.data_ptr() + 1, *([0] * 8), dgate.data_ptr(), *([0] * 8))
    assert zb._lib().zero1_block_norm_backward(c, io, None, 0, zb._launch_stream(None)) == 0
    assert (dgate == 0.0).all()
