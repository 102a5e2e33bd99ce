"""Sigmoid gates of every size, in fp32, without norms around them, so that the
factor and its slope are seen alone.

Bounds, in half ulps u = 2^-24 of the result: the factor is 1 / (1 + e) or
e / (1 + e), e = exp(-|x|): an exponential of 2.5 ulps = 5u, 1 + e one u, a
reciprocal of up to 2 ulps = 4u, the product u, in all 11u; the residual scale,
the product with y and the store 3u more: 16u.  The slope e / (1 + e)^2: 5u, twice
5u, two products, and four roundings around it: 24u.  Below 1e-37 (block_reference.TINY) fp32 has
fewer bits."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
import block_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
EDGES = [0.0, -0.0, 1e-30, 1e-3, 0.5, 3.0, 6.0, 10.0, 16.0, 17.0, 17.5, 20.0, 40.0, 60.0, 80.0, 85.0, 87.0, 88.0, 88.8, 90.0,
         100.0, 104.0, 127.0, 128.0, 200.0, 1e4, 3e38]


def gates(n, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, generator=g, dtype=F32) * 40
    e = torch.tensor(EDGES + [-v for v in EDGES])
    x[:min(n, e.numel())] = e[:n]
    return x.to(dtype)


def close(got, want, ulps, what):
    got, want = got.double().cpu(), want.double()
    bad = ~((got - want).abs() <= want.abs() * ulps * ref.U + ref.TINY)
    if bad.any():
        j = bad.flatten().nonzero()[0].item()
        raise AssertionError(f"{what}: {int(bad.sum())} outside, first {got.flatten()[j].item()!r} for "
                             f"{want.flatten()[j].item()!r}")


def exact(x):
    """The factor and its slope in 64 bits, without 1 - s."""
    x = x.double()
    return torch.sigmoid(x), torch.sigmoid(x) * torch.sigmoid(-x)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,D", [(2, 512), (3, 250), (1, 4096), (2, 9000), (700, 96)])
@pytest.mark.parametrize("kind", ["channel", "token", "full"])
def test_factor_and_slope(cuda_device, dtype, T, D, kind):
    g = torch.Generator().manual_seed(T + D)
    shape = {"channel": (D,), "token": (T, 1), "full": (T, D)}[kind]
    gate = gates(shape[0] * (shape[1] if len(shape) == 2 else 1), 5, dtype).view(shape)
    y, dr = (torch.randn((T, D), generator=g).abs() + 0.1 for _ in range(2))   # of one sign: sums do not cancel
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    cfg = z.BlockNorm(residual_scale=0.5, gate_act="sigmoid")
    s, slope = exact(gate)
    r = torch.empty((T, D), device=cuda_device)
    z.zero1_block_norm_forward(cfg, dev(y), torch.zeros_like(r), r, gate=dev(gate))
    close(r, 0.5 * s * y.double(), 16, "r")
    dx, dy = torch.empty_like(r), torch.empty_like(r)
    dgate = torch.empty(shape, dtype=dtype if kind == "full" else F32, device=cuda_device)
    z.zero1_block_norm_backward(cfg, None, dev(dr), dev(y), None, None, None, dy, dx, gate=dev(gate), dgate=dgate)
    assert torch.equal(dx.cpu(), dr)
    close(dy, 0.5 * s * dr.double(), 16, "dy")
    p = 0.5 * dr.double() * y.double()
    want = {"channel": lambda: p.sum(0) * slope, "token": lambda: p.sum(1, keepdim=True) * slope,
            "full": lambda: p * slope}[kind]()
    if dgate.dtype == BF16:
        ulps = 2 ** 16 + 32                # rounded to bf16: half an ulp is 2^-8
    else:
        ulps = 24 + {"channel": T, "token": D, "full": 0}[kind]   # a sum of n terms of one sign: n u
    close(dgate, want, ulps, "dgate")


@pytest.mark.parametrize("kind", ["channel", "token", "full"])
def test_infinite_and_nan_gates(cuda_device, kind):
    """sigmoid(+-Inf) is 1 or 0 with slope 0; a NaN stays where it is."""
    T, D = 3, 256
    gate = torch.zeros({"channel": (D,), "token": (T, 1), "full": (T, D)}[kind])
    flat = gate.view(-1)
    flat[0], flat[1], flat[2] = float("inf"), float("-inf"), float("nan")
    y = torch.ones((T, D))
    dev = lambda t: t.to(cuda_device)  # noqa: E731
    cfg = z.BlockNorm(gate_act="sigmoid")
    r = torch.empty((T, D), device=cuda_device)
    z.zero1_block_norm_forward(cfg, dev(y), torch.zeros_like(r), r, gate=dev(gate))
    assert torch.equal(torch.nan_to_num(r.cpu(), nan=7.0), torch.nan_to_num(torch.sigmoid(gate) * y, nan=7.0))
    dx, dy, dgate = torch.empty_like(r), torch.empty_like(r), torch.empty_like(dev(gate))
    z.zero1_block_norm_backward(cfg, None, dev(y), dev(y), None, None, None, dy, dx, gate=dev(gate), dgate=dgate)
    assert torch.equal(torch.nan_to_num(dy.cpu(), nan=7.0), torch.nan_to_num(torch.sigmoid(gate) * y, nan=7.0))
    d = dgate.cpu().view(-1)
    assert d[0] == 0 and d[1] == 0 and torch.isnan(d[2]) and (d[3:] > 0).all()
