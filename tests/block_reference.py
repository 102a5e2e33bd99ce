"""The training-block operators in 64 bits, written from their formulas, with
the error bounds that the tests hold the kernels to.

Bounds: u = 2^-24 is half an fp32 ulp, relative.  A sum of n products in any
order is within (n + 2) u of the sum of the terms' magnitudes.  Rounding a
result to bf16 adds at most 2^-8 of its magnitude (half an ulp), to fp32 u.
"""
import torch

U = 2.0 ** -24
BF16_HALF_ULP = 2.0 ** -8
TINY = 1e-37                # below it fp32 (and bf16) rounds to a fixed step
SIGMOID = 16 * 2.0 ** -23   # the fast exponential and division, |gate| <= 6: 9 + 2 ulp, with margin
BLOCK = 128


def up(n, m=BLOCK):
    return -(-n // m) * m


def half_ulp(dtype):
    return BF16_HALF_ULP if dtype == torch.bfloat16 else U


def scale_exponent(amax):
    """The least e in [-119, 119] with amax <= 448 * 2^e, by search."""
    e = torch.full(amax.shape, 119, dtype=torch.int64)
    for k in range(118, -120, -1):
        e = torch.where(amax <= 448.0 * 2.0 ** k, torch.full_like(e, k), e)
    return e


def pack(x):
    """(codes, biased exponents [rows, blocks]) of an fp64 [T, K] matrix."""
    T, K = x.shape
    v = torch.zeros((T, up(K)), dtype=torch.float64)
    v[:, :K] = x
    v = v.view(T, -1, BLOCK)
    bad = ~torch.isfinite(v).all(dim=2)
    v = torch.where(bad[:, :, None], torch.zeros_like(v), v)
    e = scale_exponent(v.abs().amax(dim=2))
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # the codes 0 .. 448 in order
    q = (v.abs() * (2.0 ** (-e.double()))[:, :, None]).clamp(max=448.0)
    hi = torch.searchsorted(grid, q).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    to_lo, to_hi = q - grid[lo], grid[hi] - q
    pick = torch.where((to_lo < to_hi) | ((to_lo == to_hi) & (lo % 2 == 0)), lo, hi)
    codes = pick.to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 7)
    codes = torch.where(bad[:, :, None], torch.zeros_like(codes), codes)
    exps = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return codes.view(T, -1), exps


def values(codes, exps, K):
    """fp64 values of codes [T, Kp] with exponents [T, blocks]."""
    T = codes.shape[0]
    b = codes.long()
    f, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(f == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (f - 7).double())
    s = torch.where(exps == 255, torch.full(exps.shape, float("nan"), dtype=torch.float64),
                    2.0 ** (exps.long() - 127).double())
    v = torch.where(b >= 128, -mag, mag).view(T, -1, BLOCK) * s[:, :, None]
    return v.view(T, -1)[:, :K]


def gate_factor(gate, act):
    if gate is None:
        return torch.ones((), dtype=torch.float64)
    return torch.sigmoid(gate) if act == "sigmoid" else gate


def forward(y, x, w_post, w_pre, gate, act, alpha, eps):
    """All fp64; None leaves a norm or the gate out.  Differentiable."""
    f = {"yh": y, "rstd_post": None, "rstd_pre": None, "h": None, "rh": None}
    u = y
    if w_post is not None:
        f["rstd_post"] = (y.square().mean(1) + eps).rsqrt()
        f["yh"] = y * f["rstd_post"][:, None]
        u = f["yh"] * w_post
    f["r"] = x + alpha * gate_factor(gate, act) * u
    if w_pre is not None:
        f["rstd_pre"] = (f["r"].square().mean(1) + eps).rsqrt()
        f["rh"] = f["r"] * f["rstd_pre"][:, None]
        f["h"] = f["rh"] * w_pre
    return f


def backward(dh, dr, yh, rh, rstd_post, rstd_pre, w_post, w_pre, gate, act, alpha):
    """The gradients and, as *_mag, what their rounding errors scale with."""
    D = yh.shape[1]
    g = gate_factor(gate, act)
    o = {"dw_post": None, "dw_pre": None, "dgate": None}
    d = torch.zeros_like(yh) if dr is None else dr
    dmag = d.abs()
    if w_pre is not None:
        o["dw_pre"], o["dw_pre_mag"] = (dh * rh).sum(0), (dh * rh).abs().sum(0)
        wdh = dh * w_pre
        mean, mmag = (wdh * rh).mean(1, keepdim=True), (wdh * rh).abs().mean(1, keepdim=True)
        s = rstd_pre[:, None]
        d = d + s * (wdh - rh * mean)
        dmag = dmag + s * (wdh.abs() * 4 + rh.abs() * mmag * (D + 8))
    o["dx"], o["dx_mag"] = d, dmag
    u = yh * w_post if w_post is not None else yh
    p, pmag = alpha * d * u, abs(alpha) * dmag * u.abs()
    if gate is not None:
        slope = g * (1 - g) if act == "sigmoid" else torch.ones_like(g)
        dims = {1: 0, 2: 1}[gate.dim()] if gate.shape != yh.shape else None
        keep = gate.dim() == 2
        o["dgate"] = (p if dims is None else p.sum(dims, keepdim=keep)) * slope
        o["dgate_mag"] = (pmag if dims is None else pmag.sum(dims, keepdim=keep)) * slope
    dyh, dyh_mag = alpha * g * d, (alpha * g).abs() * dmag
    o["dy"], o["dy_mag"] = dyh, dyh_mag
    if w_post is not None:
        o["dw_post"], o["dw_post_mag"] = (dyh * yh).sum(0), (dyh_mag * yh.abs()).sum(0)
        wd, wmag = dyh * w_post, dyh_mag * w_post.abs()
        s = rstd_post[:, None]
        o["dy"] = s * (wd - yh * (wd * yh).mean(1, keepdim=True))
        o["dy_mag"] = s * (wmag * 4 + yh.abs() * (wmag * yh.abs()).mean(1, keepdim=True) * (D + 8))
    return o
