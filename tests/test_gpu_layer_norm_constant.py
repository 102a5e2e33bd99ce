"""Layer norm of constant rows: the mean is the constant itself, whatever the
width, and nothing is left of r - mean to be divided by the square root of eps."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("D", [64, 1000, 1021, 1023, 4095, 4096, 5000, 7000, 9183, 12072, 16320])
@pytest.mark.parametrize("act,res", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("residual", [False, True])
def test_constant_rows(D, act, res, residual):
    # eight bits each: their sums over up to 2^14 columns are exact in fp32
    values = [k * s for k in range(128, 256, 3) for s in (2.0 ** -9, 1.0, -8.0)]
    x = torch.tensor(values, device="cuda").to(res)[:, None].expand(-1, D).contiguous()
    T = x.shape[0]
    b = torch.randn(D, device="cuda").to(act)
    h, mean, rstd = torch.full((T, D), 7.0, dtype=act, device="cuda"), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y = torch.zeros(T, D, dtype=act, device="cuda") if residual else None
    z.zero1_layer_norm_forward(z.LayerNorm(eps=1e-5), x, h, mean, rstd, w=torch.full_like(b, 3.0), b=b, y=y,
                               r=torch.empty_like(x) if residual else None)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(h, b.expand(T, D))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=4 * 2.0 ** -23, atol=0)


@pytest.mark.parametrize("D", [64, 1000, 1021, 9183, 16384])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_row_that_is_not_finite_keeps_its_mean(D, bad):
    x = torch.ones(3, D, device="cuda")
    x[1, D // 2] = bad
    h, mean, rstd = torch.empty_like(x), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    z.zero1_layer_norm_forward(z.LayerNorm(), x, h, mean, rstd)
    assert mean.tolist()[::2] == [1.0, 1.0] and bool((h[::2] == 0).all())
    assert mean[1].item() == bad or (bad != bad and bool(torch.isnan(mean[1])))
    assert bool(torch.isnan(h[1]).all())
