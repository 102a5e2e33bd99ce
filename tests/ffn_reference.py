"""The gated feed-forward block in float64, with the first-order bounds that its
fp32 sums and bf16 results obey."""
import math

import torch

A, B = math.sqrt(2.0 / math.pi), 0.044715
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
# The largest slopes of act and of act' (silu: 1.0999 and 0.5; gelu: 1.1290 and 0.8142).
SLOPE, CURVE = 1.13, 0.82
TINY = 2.0 ** -126


HALF_STEP = 2.0 ** -24


def own(g: torch.Tensor, act: str):
    """What the activation's own arithmetic in fp32 adds: the relative error of f = g
    s(k) and the absolute one of f' = s + g k' (s - s^2).  k by up to four roundings
    and t = k log2 e by one more, of a constant that is rounded too: 6 half steps of k,
    which 2^t turns into 6 |k| half steps of e; 2^t itself 4.  In s = e / (1 + e) an error
    of e counts 1 - s times; 1 + e, 1 / x and the product are good for 6 half steps, none
    where t is cut at 64 and all three are exact.  s - s^2 moves with s by at most 1 times
    and is rounded once, as are its product and the sum."""
    k = g if act == "silu" else 2 * A * (g + B * g.pow(3))
    gdk = g if act == "silu" else 2 * A * (g + 3 * B * g.pow(3))
    s, rest = torch.sigmoid(k), torch.sigmoid(-k)
    es = ((6 * k.abs().clamp(max=110) + 4) * rest + torch.where(k > 44.5, 0.0, 6.0)) * HALF_STEP
    slope = s * rest
    edf = s * es + gdk.abs() * (s * es + HALF_STEP * slope) + 8 * HALF_STEP * (s + gdk.abs() * slope)
    return es + 2 * HALF_STEP, 1.01 * edf


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
    ef = SLOPE * eg + own(g, act)[0] * (f.abs() + TINY)
    a = f * u
    return a, ef * u.abs() + (f.abs() + ef) * eu + HALF[torch.bfloat16] * a.abs() * 1.01 + 2.0 ** -133


def backward(da, h, w_gate, w_up, act):
    """(dg, bound), (du, bound)."""
    (g, eg), (u, eu) = projections(h, w_gate), projections(h, w_up)
    f, df = activation(g, act)
    d = da.double()
    rel, edf = own(g, act)
    ef = SLOPE * eg + rel * (f.abs() + TINY)
    edf = CURVE * eg + edf
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
    """dy^T x (+ start) and the bound; fp32 results in runs of 512 rows, bf16 ones of
    131072, whose sums are added with one rounding each."""
    y, x = dy.double(), x.double()
    dw, size = y.t() @ x, y.abs().t() @ x.abs()
    run = 512 if dtype is torch.float32 else 131072
    e = sum_bound(min(dy.shape[0], run), size) + -(-dy.shape[0] // run) * 2.0 ** -24 * size
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
