"""The gated feed-forward block in float64, with the first-order bounds that its
fp32 sums and bf16 results obey."""
import math

import torch

A, B = math.sqrt(2.0 / math.pi), 0.044715
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# The largest slopes of act and of act' (silu: 1.0999 and 0.5; gelu: 1.1290 and 0.8142).
SLOPE, CURVE = 1.13, 0.82
# The activation's own arithmetic in fp32: k(g) by three roundings, its logistic
# function and slope within 16 half steps, three more products.
OWN = 32 * 2.0 ** -24
TINY = 2.0 ** -126


def sum_bound(terms: int, size: torch.Tensor) -> torch.Tensor:
    """Error of a sum of `terms` exact products of total magnitude `size` on the
    tensor cores: at most one step (2^-23, they truncate) of the partial sum's
    magnitude for every 16 terms, and as much for aligning the 16 products and
    for the few additions of partial sums."""
    return (2 * (terms / 16 + 1) + 20) * 2.0 ** -23 * size


def activation(g: torch.Tensor, act: str):
    """act(g) and act'(g)."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1.0 + g * torch.sigmoid(-g))
    t = torch.tanh(A * (g + B * g.pow(3)))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * A * (1.0 + 3.0 * B * g * g)


def projections(h, w):
    """h w^T and the bound of its error."""
    h, w = h.double(), w.double()
    return h @ w.t(), sum_bound(h.shape[1], h.abs() @ w.abs().t())


def forward(h, w_gate, w_up, act):
    """a and the bound of its error."""
    (g, eg), (u, eu) = projections(h, w_gate), projections(h, w_up)
    f, _ = activation(g, act)
    ef = SLOPE * eg + OWN * (f.abs() + TINY)
    a = f * u
    return a, ef * u.abs() + (f.abs() + ef) * eu + HALF[torch.bfloat16] * a.abs() * 1.01 + 2.0 ** -133


def backward(da, h, w_gate, w_up, act):
    """(dg, bound), (du, bound)."""
    (g, eg), (u, eu) = projections(h, w_gate), projections(h, w_up)
    f, df = activation(g, act)
    d = da.double()
    ef = SLOPE * eg + OWN * (f.abs() + TINY)
    # act' is a sum of s and g s (1 - s) k', each within OWN of itself; |g| s (1 - s) k' is at most 1.2
    edf = CURVE * eg + OWN * 2.2
    dg, du = d * u * df, d * f
    r = 1.01 * HALF[torch.bfloat16]
    return ((dg, d.abs() * (edf * u.abs() + (df.abs() + edf) * eu) + r * dg.abs() + 2.0 ** -133),
            (du, d.abs() * ef + r * du.abs() + 2.0 ** -133))


def input_grad(dg, du, w_gate, w_up):
    dg, du, g, u = dg.double(), du.double(), w_gate.double(), w_up.double()
    dh = dg @ g + du @ u
    size = dg.abs() @ g.abs() + du.abs() @ u.abs()
    return dh, sum_bound(2 * dg.shape[1], size) + 1.01 * HALF[torch.bfloat16] * dh.abs() + 2.0 ** -133


def weight_grad(dy, x, dtype, start=None):
    """dy^T x (+ start) and the bound; fp32 results in runs of 2048 rows, whose
    sums are added with one rounding each."""
    y, x = dy.double(), x.double()
    dw, size = y.t() @ x, y.abs().t() @ x.abs()
    runs = max(1, -(-dy.shape[0] // 2048)) if dtype is torch.float32 else 1
    e = sum_bound(min(dy.shape[0], 2048) if dtype is torch.float32 else dy.shape[0], size) + runs * 2.0 ** -24 * size
    if start is not None:
        dw = dw + start.double()
    return dw, e + 1.01 * HALF[dtype] * (dw.abs() + e) + 2.0 ** -133


def check(got: torch.Tensor, want_bound, what: str) -> None:
    want, bound = want_bound
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    if bad.any():
        k = int((off / bound).nan_to_num(float("inf")).argmax())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off their bound; the worst, at {k}: "
                             f"{got.flatten()[k].item()!r} for {want.flatten()[k].item()!r}, "
                             f"{(off / bound).flatten()[k].item():.3g} times the bound")
