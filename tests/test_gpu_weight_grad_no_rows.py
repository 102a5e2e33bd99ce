"""Weight gradients without rows: +0, or, accumulated into, every bit as it was."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
BITS = {BF16: torch.int16, F32: torch.int32}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,K", [(1, 1), (5, 7), (300, 264)])
def test_bf16_weight_grad(dtype, N, K):
    g = torch.Generator(device="cuda").manual_seed(N)
    info = torch.iinfo(BITS[dtype])
    dw = torch.randint(info.min, info.max, (N, K), generator=g, device="cuda", dtype=BITS[dtype])  # (NaNs of every kind)
    dw[0, 0] = info.min  # -0
    start = dw.clone()
    dy, x = torch.empty(0, N, dtype=BF16, device="cuda"), torch.empty(0, K, dtype=BF16, device="cuda")
    z.zero1_weight_grad_bf16(dy, x, dw.view(dtype), accumulate=True)
    assert torch.equal(dw, start)
    z.zero1_weight_grad_bf16(dy, x, dw.view(dtype))
    assert not bool(dw.any())
