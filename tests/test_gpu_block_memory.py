"""Where the training-block operators' buffers live: pinned host tensors where
they are allowed, workspaces always in device memory, refusals elsewhere."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
from zero_sharded_mixed_zero1_gb300 import block as zb
import test_gpu_block_ops as ops

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def pinned_like(t, cuda, pad=0, off=0):
    """ops.dev in pinned host memory."""
    return None if t is None else t.contiguous().pin_memory()


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("D", [768, 1021])
@pytest.mark.parametrize("side", [False, True])
def test_backward_on_pinned_tensors_equals_device_tensors(cuda_device, monkeypatch, ckpt, D, side):
    """The workspace of the weights' gradients is device memory although every
    tensor of the call is in host memory, on either kind of stream argument."""
    p = ops.Problem(1500, D, BF16, BF16, True, True, "channel", "sigmoid", seed=30)
    want, _ = ops.run_backward(p, cuda_device, ckpt)
    taken = []
    real = zb._workspace

    def spy(workspace, nbytes, stream):
        got = real(workspace, nbytes, stream)
        taken.append(got[2])
        return got
    monkeypatch.setattr(zb, "_workspace", spy)
    monkeypatch.setattr(ops, "dev", pinned_like)
    if side:
        st = torch.cuda.Stream()
        backward = z.zero1_block_norm_backward
        monkeypatch.setattr(z, "zero1_block_norm_backward", lambda *a, **k: backward(*a, stream=st.cuda_stream, **k))
        torch.cuda.synchronize()
    got, _ = ops.run_backward(p, cuda_device, ckpt)
    torch.cuda.synchronize()
    assert taken and all(t.is_cuda for t in taken)
    for k in want:
        assert torch.equal(got[k].cpu(), want[k].cpu()), k


def test_a_host_workspace_is_refused(cuda_device, monkeypatch):
    host = torch.zeros(1 << 24, dtype=torch.uint8).pin_memory()
    p = ops.Problem(50, 768, BF16, BF16, True, True, "channel", "linear", seed=31)
    with pytest.raises(ValueError, match="CUDA uint8"):
        z.zero1_weight_grad(torch.zeros((8, 8), dtype=BF16, device=cuda_device), z.new_checkpoint(8, 8, cuda_device),
                            torch.zeros((8, 8), device=cuda_device), workspace=host)
    monkeypatch.setattr(zb, "_workspace", lambda w, n, s: (host.data_ptr(), host.numel(), host))  # as a C caller may
    with pytest.raises(z.Zero1Error, match="device memory"):
        ops.run_backward(p, cuda_device, True)
    x, dy, _ = ops.weight_grad_problem(100, 771, 200)     # rows of 771 need an aligned copy in the workspace
    k = z.new_checkpoint(100, 200, cuda_device)
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    with pytest.raises(z.Zero1Error, match="device memory"):
        z.zero1_weight_grad(dy.to(cuda_device), k, torch.zeros((771, 200), device=cuda_device))
    assert (host == 0).all()


def test_weight_grad_refuses_host_tensors(cuda_device):
    x, dy, col = ops.weight_grad_problem(64, 64, 128)
    k = z.new_checkpoint(64, 128, cuda_device)
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    dw = torch.zeros((64, 128), device=cuda_device)
    for args, kw in (((dy.pin_memory(), k, dw), {}), ((dy.to(cuda_device), k, dw.cpu().pin_memory()), {}),
                     ((dy.to(cuda_device), k, dw), dict(col_scale=col.pin_memory()))):
        with pytest.raises(z.Zero1Error, match="device memory"):
            z.zero1_weight_grad(*args, **kw)
    empty = z.new_checkpoint(0, 128, cuda_device)
    with pytest.raises(z.Zero1Error, match="device memory"):
        z.zero1_weight_grad(torch.empty((0, 64), dtype=BF16, device=cuda_device), empty, dw.cpu().pin_memory())
