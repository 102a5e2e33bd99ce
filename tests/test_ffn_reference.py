"""The feed-forward block's reference in 64 bits, on the CPU: against automatic
differentiation and differences; its bounds hold for fp32 arithmetic rounded to
bf16 and refuse planted mistakes."""
import pytest
import torch

import ffn_reference as ref

BF16 = torch.bfloat16


def tensors(T=7, D=40, F=24):
    g = torch.Generator().manual_seed(1)
    r = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(BF16)  # noqa: E731
    return r(T, D), r(F, D, std=D ** -0.5), r(F, D, std=D ** -0.5), r(T, F, std=1e-2)


def block(h, wg, wu, act):
    g = h @ wg.t()
    f = torch.nn.functional.silu(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    return f * (h @ wu.t())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_against_automatic_differentiation(act):
    h, wg, wu, da = tensors()
    hd, gd, ud = (t.double().requires_grad_() for t in (h, wg, wu))
    a = block(hd, gd, ud, act)
    a.backward(da.double())
    assert torch.allclose(ref.forward(h, wg, wu, act)[0], a.detach(), rtol=1e-13, atol=0)
    (dg, _), (du, _) = ref.backward(da, h, wg, wu, act)
    assert torch.allclose(dg @ wg.double() + du @ wu.double(), hd.grad, rtol=1e-10, atol=1e-16)
    assert torch.allclose(dg.t() @ h.double(), gd.grad, rtol=1e-10, atol=1e-16)
    assert torch.allclose(du.t() @ h.double(), ud.grad, rtol=1e-10, atol=1e-16)
    x, y = dg.to(BF16), du.to(BF16)
    assert torch.equal(ref.input_grad(x, y, wg, wu)[0], x.double() @ wg.double() + y.double() @ wu.double())
    assert torch.equal(ref.weight_grad(x, h, torch.float32)[0], x.double().t() @ h.double())


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_slopes_against_differences(act):
    g = torch.linspace(-12, 12, 481, dtype=torch.float64)
    f, df = ref.activation(g, act)
    step = 1e-5
    want = (ref.activation(g + step, act)[0] - ref.activation(g - step, act)[0]) / (2 * step)
    assert (df - want).abs().max() < 1e-9  # a third derivative of at most 3 times step^2 / 6, and 1e-15 * 12 / step
    assert df.abs().max() <= ref.SLOPE
    assert ((ref.activation(g + step, act)[1] - ref.activation(g - step, act)[1]) / (2 * step)).abs().max() <= ref.CURVE


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_the_bounds_hold_for_fp32_and_refuse_mistakes(act):
    h, wg, wu, da = tensors(T=64, D=256, F=96)
    g, u = h.float() @ wg.float().t(), h.float() @ wu.float().t()
    f, df = (t.float() for t in ref.activation(g, act))
    d = da.float()
    want_a = ref.forward(h, wg, wu, act)
    want_dg, want_du = ref.backward(da, h, wg, wu, act)
    ref.check((f * u).to(BF16), want_a, "a")
    ref.check((d * u * df).to(BF16), want_dg, "dg")
    ref.check((d * f).to(BF16), want_du, "du")
    other = "gelu" if act == "silu" else "silu"
    wrong = [((f * u).to(BF16) * 1.02, want_a), ((g * u).to(BF16), want_a), ((ref.activation(g, other)[0] * u).to(BF16), want_a),
             ((d * u).to(BF16), want_dg), ((d * f * df).to(BF16), want_dg), ((d * g).to(BF16), want_du),
             ((d * f).roll(1, 0).to(BF16), want_du)]
    for got, want in wrong:
        with pytest.raises(AssertionError):
            ref.check(got, want, "planted")
