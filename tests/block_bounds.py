"""Rounding-error bounds of the block norms, to first order: every rounding of
the kernels' fp32 arithmetic is carried to the results by the formulas, and the
terms are added.  On any device.

u = 2^-24, half an fp32 ulp, relative.  A sum of n terms in any order is within
(n + 2) u of the sum of their magnitudes (n u for the additions, 2 u for products
and scale).  Products of second order are covered by the small constants.  All
bounds are those of the value before it is stored; storing adds half an ulp of
the type (block_reference.half_ulp)."""
import torch

import block_reference as ref
from block_reference import U

GATE = 16 * U      # of a sigmoid gate's factor, relative (11 u), and its slope (18 u with the product after it below)
SLOPE = 24 * U


def _mean(t):
    return t.mean(1, keepdim=True)


def forward_bounds(f, w_post, w_pre, gate, act, alpha, eps, D):
    """Errors of r, h, rstd_post, rstd_pre and, relative, of yh and rh."""
    o = {}
    stat = (D + 8) * U                    # a mean of D squares and its reciprocal root, relative
    g = ref.gate_factor(gate, act)
    u = f["yh"] if w_post is None else f["yh"] * w_post
    if w_post is not None:
        o["rstd_post"] = f["rstd_post"] * stat
    o["yh_rel"] = stat if w_post is not None else 0.0
    o["r"] = (alpha * g * u).abs() * (o["yh_rel"] + 4 * U + (GATE if act == "sigmoid" else 0.0)) + f["r"].abs() * U
    if w_pre is not None:
        rel = stat + (f["r"].abs() * o["r"]).mean(1) / (f["r"].square().mean(1) + eps)
        o["rstd_pre"] = f["rstd_pre"] * rel
        o["rh_rel"], o["rh_abs"] = rel[:, None] + 2 * U, o["r"] * f["rstd_pre"][:, None]
        o["h"] = f["h"].abs() * (rel[:, None] + 3 * U) + o["rh_abs"] * w_pre.abs()
    return o


def backward_bounds(want, dh, dr, yh, rh, rstd_post, rstd_pre, w_post, w_pre, gate, act, alpha):
    """Errors of dx, dy, dw_post, dw_pre and dgate, given the exact results."""
    T, D = yh.shape
    o = {}
    x, xe = want["dx"], want["dx"].abs() * 2 * U
    if w_pre is not None:
        wdh = dh * w_pre
        m, mags = _mean(wdh * rh), _mean((wdh * rh).abs())
        xe = xe + rstd_pre[:, None].abs() * (wdh.abs() * 4 * U + rh.abs() * (mags * (D + 6) * U + m.abs() * 4 * U))
        o["dw_pre"] = (dh * rh).abs().sum(0) * (T + 6) * U
    o["dx"] = xe
    g, ge = ref.gate_factor(gate, act), GATE if act == "sigmoid" and gate is not None else 0.0
    u = yh if w_post is None else yh * w_post
    if gate is not None:
        p = alpha * x * u
        pe = (alpha * u).abs() * xe + p.abs() * 4 * U
        if gate.shape == yh.shape:
            o["dgate"] = pe
        else:
            dim, n = (0, T) if gate.dim() == 1 else (1, D)
            keep = gate.dim() == 2
            o["dgate"] = pe.sum(dim, keepdim=keep) + p.abs().sum(dim, keepdim=keep) * (n + 4) * U
        if act == "sigmoid":
            o["dgate"] = o["dgate"] * (g * (1 - g)) + want["dgate"].abs() * SLOPE
    d = alpha * g * x                     # the gradient of u
    de = (alpha * g).abs() * xe + d.abs() * (3 * U + ge)
    if w_post is None:
        o["dy"] = de
        return o
    o["dw_post"] = (de * yh.abs()).sum(0) + (d * yh).abs().sum(0) * (T + 6) * U
    wd, we = d * w_post, de * w_post.abs() + (d * w_post).abs() * U
    m = _mean(wd * yh)
    me = _mean(we * yh.abs()) + _mean((wd * yh).abs()) * (D + 10) * U
    s = rstd_post[:, None].abs()
    o["dy"] = s * (we + wd.abs() * 4 * U + yh.abs() * (me + m.abs() * 4 * U)) + want["dy"].abs() * 2 * U
    return o


def outside(got, want, err, dtype):
    """Which elements are further off than their error and the type's rounding."""
    return ~((got.double() - want).abs() <= err + (want.abs() + err) * ref.half_ulp(dtype) + ref.TINY)
