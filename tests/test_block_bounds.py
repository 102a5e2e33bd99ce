"""The bounds that the block norms are held to (block_bounds.py), without a GPU:
fp32 arithmetic of the same formulas stays within them, and results with a
mistake in them do not."""
import pytest
import torch

import block_bounds as bb
import block_reference as ref

BF16, F32 = torch.bfloat16, torch.float32
SIZES = [(5, 7), (4, 512), (6, 768), (4, 1021), (3, 4096), (3, 8192), (2, 16384)]


def problem(T, D, gate, act, seed=0):
    """Inputs on the fp32 grid; the gradients lie along the rows, so that the
    rows' means matter."""
    g = torch.Generator().manual_seed(seed + T + D)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    y, x = r(T, D) * 0.7, r(T, D) * 2
    shape = {None: None, "channel": (D,), "token": (T, 1), "full": (T, D)}[gate]
    p = {"y": y, "x": x, "w_post": 1 + 0.1 * r(D), "w_pre": 1 + 0.2 * r(D),
         "gate": None if shape is None else 0.5 + 0.7 * r(*shape), "dh": 1e-2 * (r(T, D) + x), "dr": 1e-2 * (r(T, D) + y)}
    p = {k: None if t is None else t.double() for k, t in p.items()}
    f = ref.forward(p["y"], p["x"], p["w_post"], p["w_pre"], p["gate"], act, 0.5, 1e-6)
    p["yh"], p["rh"] = f["yh"].float().double(), f["rh"].float().double()
    p["rstd_post"], p["rstd_pre"] = f["rstd_post"].float().double(), f["rstd_pre"].float().double()
    return p


ARGS = ("dh", "dr", "yh", "rh", "rstd_post", "rstd_pre", "w_post", "w_pre", "gate")


def results(p, act, dtype=torch.float64):
    return ref.backward(*(None if p[k] is None else p[k].to(dtype) for k in ARGS), act, 0.5)


@pytest.mark.parametrize("T,D", SIZES)
@pytest.mark.parametrize("gate,act", [(None, "linear"), ("channel", "sigmoid"), ("token", "linear"), ("token", "sigmoid"),
                                      ("full", "sigmoid"), ("channel", "linear")])
def test_fp32_arithmetic_is_within(T, D, gate, act):
    p = problem(T, D, gate, act)
    want = results(p, act)
    err = bb.backward_bounds(want, *(p[k] for k in ARGS), act, 0.5)
    got = results(p, act, F32)
    for k in ("dx", "dy", "dw_post", "dw_pre", "dgate"):
        if want[k] is None:
            continue
        for dtype in (F32, BF16):
            assert not bb.outside(got[k].to(dtype), want[k], err[k], dtype).any(), (k, dtype)


def mistakes(p, want, gate, act):
    """name -> (result, wrong values of it)."""
    g, a = ref.gate_factor(p["gate"], act), 0.5
    d = a * g * want["dx"]
    s, wd = p["rstd_post"][:, None], d * p["w_post"]
    mean = (wd * p["yh"]).mean(1, keepdim=True)
    plain = p["dr"] + p["rstd_pre"][:, None] * (p["dh"] * p["w_pre"])
    yield "dy is zero", "dy", torch.zeros_like(want["dy"])
    yield "dy without its mean term", "dy", s * wd
    yield "dy with the other sign of it", "dy", s * (wd + p["yh"] * mean)
    yield "dy with the mean over one column too many", "dy", s * (wd - p["yh"] * mean * (1 - 1 / (p["yh"].shape[1] + 1)))
    yield "dy with another row's mean", "dy", s * (wd - p["yh"] * mean.roll(1, 0))
    yield "dy with another row's statistic", "dy", want["dy"] / s * s.roll(1, 0)
    yield "dy without the weight", "dy", s * (d - p["yh"] * (d * p["yh"]).mean(1, keepdim=True))
    yield "dy from a dx without its mean", "dy", s * (a * g * plain * p["w_post"] -
                                                      p["yh"] * (a * g * plain * p["w_post"] * p["yh"]).mean(1, keepdim=True))
    yield "dx without its mean term", "dx", plain
    yield "dx without dr", "dx", want["dx"] - p["dr"]
    yield "dw_post without the last row", "dw_post", (d * p["yh"])[:-1].sum(0)
    yield "dw_pre without the last row", "dw_pre", (p["dh"] * p["rh"])[:-1].sum(0)
    if gate is not None:
        yield "dgate without the scale", "dgate", want["dgate"] / a
        yield "dw_post without the gate", "dw_post", (a * want["dx"] * p["yh"]).sum(0)
        if act == "sigmoid":
            yield "dgate without the slope", "dgate", want["dgate"] / (g * (1 - g))


@pytest.mark.parametrize("T,D", SIZES[1:])
@pytest.mark.parametrize("gate,act", [(None, "linear"), ("channel", "linear"), ("token", "sigmoid"), ("full", "sigmoid")])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_mistakes_are_outside(T, D, gate, act, dtype):
    p = problem(T, D, gate, act, seed=1)
    want = results(p, act)
    err = bb.backward_bounds(want, *(p[k] for k in ARGS), act, 0.5)
    for what, k, wrong in mistakes(p, want, gate, act):
        if "one column too many" in what and (dtype == BF16 or D > 1021):
            continue    # 1 / (D + 1) of the mean is below bf16's rounding, or the bound of a sum in any order
        assert bb.outside(wrong.to(dtype), want[k], err[k], dtype).any(), what


@pytest.mark.parametrize("T,D", SIZES)
def test_a_bound_is_a_few_percent_of_its_result_at_most(T, D):
    """Of the results' norms; (D + 10) u is 1e-3 at 16384 columns."""
    p = problem(T, D, "channel", "linear", seed=2)
    want = results(p, "linear")
    err = bb.backward_bounds(want, *(p[k] for k in ARGS), "linear", 0.5)
    for k in ("dx", "dy", "dw_post", "dw_pre", "dgate"):
        assert err[k].norm() <= 0.02 * want[k].norm(), k
