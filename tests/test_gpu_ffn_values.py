"""The gated feed-forward block far from zero, where its activations are known
exactly: act(g) is g or 0 and its slope 1 or 0, to the last bit of a bf16 result."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
# exp(-128) is 2.6e-56, far below bf16's smallest value, and 1 + exp(-128) is 1
FAR = [128.0, 1e3, 1e5, 1e9, 1e10, 1e12, 1e13, 1.2e13, 1e16, 1.8e19, 2e19, 1e25, 1e30, 7e36, 1e38, 3.3e38]
F = 24


@pytest.fixture(autouse=True)
def no_wait_runs_out():
    yield
    assert z.zero1_device_status() == 0


def call(g, D, act):
    """(a, dg, du) for pre-activations g in every column, u = 1 and da = 0.25; D
    decides whether the contraction is split over blocks."""
    T = len(g)
    h = torch.zeros(T, D, dtype=BF16, device="cuda")
    h[:, 0], h[:, 1] = torch.tensor(g, device="cuda").to(BF16), 1.0
    wg, wu = (torch.zeros(F, D, dtype=BF16, device="cuda") for _ in range(2))
    wg[:, 0], wu[:, 1] = 1.0, 1.0
    split = z.zero1_gated_ffn_workspace("backward", T, wg, wu, h=h) > 0
    assert split == (D > 64), "the sizes are there for whole and for split tiles"
    a, dg, du = (torch.full((T, F), 7.0, dtype=BF16, device="cuda") for _ in range(3))
    z.zero1_gated_ffn_backward(torch.full_like(a, 0.25), h, wg, wu, dg, du, a=a, act=act)
    forward = torch.full_like(a, 7.0)
    z.zero1_gated_ffn_forward(h, wg, wu, forward, act=act)
    assert torch.equal(forward.view(torch.int16), a.view(torch.int16))
    return h[:, :1].float(), a.float(), dg.float(), du.float()


@pytest.mark.parametrize("D", [8, 4096])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_far_from_zero(act, D):
    g, a, dg, du = call(FAR + [-x for x in FAR], D, act)
    assert bool(torch.isfinite(g).all())
    up = (g > 0).float()
    for got, want in ((a, g * up), (dg, 0.25 * up), (du, 0.25 * g * up)):
        assert torch.equal(got, want.expand(-1, F)), (got - want)[:, 0]


@pytest.mark.parametrize("D", [8, 4096])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_rows_that_are_not_finite(act, D):
    """An Inf or a NaN in a row of h makes all of that row's results not finite (u
    is Inf times 0), NaN stays NaN, and the rows beside it are what they are alone."""
    inf, nan = float("inf"), float("nan")
    _, *got = call([1.0, inf, 2.0, -inf, -1.0, nan, 0.5], D, act)
    _, *want = call([1.0, 1.0, 2.0, 2.0, -1.0, -1.0, 0.5], D, act)
    for x, w in zip(got, want):
        assert torch.equal(x[::2], w[::2])
        assert not bool(torch.isfinite(x[[1, 3, 5]]).any())
        assert bool(torch.isnan(x[5]).all())
