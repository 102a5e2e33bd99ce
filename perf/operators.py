"""The training-block operators, as they are measured: block norms with gate
and residual scale (forward, backward), 8-bit activation checkpoints (pack,
unpack) and the weight gradient taken from a checkpoint.

A checkpoint of a [T, K] activation is a pair of uint8 tensors: `codes`
[T, Kp] (e4m3, Kp = K rounded up to 128) and `exps` [Kp / 128, Tp] (Tp = T
rounded up to 128): exps[b, t] = e + 127 is the power-of-two scale of row t's
columns [128 b, 128 b + 128), so a value is code * 2^e; 255 marks a block that
stands for NaN.  e is the smallest exponent in [-119, 119] with
max|x| <= 448 * 2^e; larger magnitudes saturate.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6
BLOCK = 128


def _up(n, m):
    return -(-n // m) * m


# ---------------------------------------------------------------- the cases --

def _norm_case(op, T, D, act, res, post, pre, gate, gate_act, ckpt, scale):
    return {"op": op, "T": T, "D": D, "act": act, "res": res, "post": post, "pre": pre, "gate": gate,
            "gate_act": gate_act, "ckpt": ckpt, "scale": scale}


def listed():
    named = [
        # one token through a block at the Llama layers' width: launch latency
        ("forward_one_token", _norm_case("forward", 1, 4096, "bf16", "bf16", True, True, "channel", "linear", True, 1.0)),
        # a micro-batch of 8192 tokens at the Llama layers' width, both checkpoints written on the way
        ("forward_block", _norm_case("forward", 8192, 4096, "bf16", "bf16", True, True, "channel", "linear", True, 0.5)),
        # an odd width, fp32 residual stream, one gate value for each token: a small model with depth gating
        ("forward_odd_f32", _norm_case("forward", 2003, 1021, "bf16", "f32", True, True, "token", "sigmoid", False, 1.0)),
        # a short batch at the GPT-2-small width from kept tensors, fp32 residual stream
        ("backward_short", _norm_case("backward", 64, 768, "bf16", "f32", True, True, "token", "linear", False, 1.0)),
        # the backward pass of forward_block from its checkpoints
        ("backward_block", _norm_case("backward", 8192, 4096, "bf16", "bf16", True, True, "channel", "linear", True, 0.5)),
        # a wide model with an elementwise sigmoid gate (an attention output gate) and long sequences
        ("backward_wide_gate", _norm_case("backward", 16384, 8192, "bf16", "bf16", True, True, "full", "sigmoid", True, 1.0)),
        # the feed-forward activation of the Llama layers kept in 8 bits
        ("pack_ffn", {"op": "pack", "T": 8192, "K": 14336, "dtype": "bf16"}),
        # an odd fp32 activation
        ("pack_odd_f32", {"op": "pack", "T": 1021, "K": 4099, "dtype": "f32"}),
        # the checkpoint of a small odd activation read back whole
        ("unpack_odd", {"op": "unpack", "T": 777, "K": 1000, "dtype": "f32"}),
        # a square projection of the Llama layers: its input's checkpoint and column scale (the norm's weight)
        ("weight_grad_square", {"op": "weight_grad", "T": 8192, "N": 4096, "K": 4096, "out": "bf16", "colscale": True}),
        # the feed-forward projection of the Llama layers: the largest product of the layer
        ("weight_grad_ffn", {"op": "weight_grad", "T": 8192, "N": 14336, "K": 4096, "out": "bf16", "colscale": True}),
        # a small odd projection with an fp32 gradient
        ("weight_grad_odd_f32", {"op": "weight_grad", "T": 777, "N": 771, "K": 1000, "out": "f32", "colscale": False}),
    ]
    return [dict(c, name=n) for n, c in named]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size of [lo, hi]: half of them multiples of 64 as models have them, half anything."""
    n = _log_int(rng, lo, hi)
    return max(lo, min(hi, _up(n, 64))) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["forward", "forward", "backward", "backward", "pack", "unpack", "weight_grad", "weight_grad"])
    if op in ("forward", "backward"):
        D = _size(rng, 64, 8192)
        T = _log_int(rng, 1, min(32768, (1 << 26) // D))
        act, res = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        gate = rng.choice(["none", "channel", "token", "full"])
        return _norm_case(op, T, D, act, res, post, pre, gate, rng.choice(["linear", "sigmoid"]),
                          rng.random() < 0.6, rng.choice([1.0, 0.5, 0.22]))
    if op in ("pack", "unpack"):
        K = _size(rng, 64, 16384)
        return {"op": op, "T": _log_int(rng, 1, min(32768, (1 << 26) // K)), "K": K,
                "dtype": rng.choice(["bf16", "f32"])}
    N, K = _size(rng, 64, 8192), _size(rng, 64, 8192)
    return {"op": op, "T": _log_int(rng, 16, min(16384, (1 << 38) // (N * K))), "N": N, "K": K,
            "out": rng.choice(["bf16", "bf16", "f32"]), "colscale": rng.random() < 0.5}


# --------------------------------------------------------------- the inputs --

def _normal(shape, std, seed, k, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + k)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _activation(T, D, std, seed, k, dtype):
    """Rows of a hidden state: normal draws with channel scales that vary, as they do."""
    x = _normal((T, D), std, seed, k)
    x *= torch.exp(_normal((D,), 0.7, seed, k + 1))
    return x.to(dtype)


def _scales_of(exps):
    """2^(exps - 127) as fp32 by its bits (NaN for 255)."""
    s = (exps.to(torch.int32) << 23).view(torch.float32)
    return torch.where(exps == 255, torch.full_like(s, float("nan")), s)


def _values(codes, exps, T, K):
    """The fp32 values that a checkpoint stands for."""
    s = _scales_of(exps[:, :T]).t().repeat_interleave(BLOCK, dim=1)
    return (codes.view(torch.float8_e4m3fn).float() * s)[:, :K].contiguous()


def _pack_plain(x):
    """codes, exps of an fp32 [T, K] tensor."""
    T, K = x.shape
    Kp, Tp = _up(K, BLOCK), _up(T, BLOCK)
    v = torch.zeros((T, Kp), device=x.device)
    v[:, :K] = x
    v = v.view(T, Kp // BLOCK, BLOCK)
    amax = v.abs().amax(dim=2)
    bad = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(bad, torch.zeros_like(amax), amax))  # amax = m 2^e, 0.5 <= m < 1
    e = (e - 9 + (m > 0.875).int()).clamp(-119, 119)                    # 448 = 0.875 * 2^9
    inv = ((127 - e) << 23).view(torch.float32)
    q = (v * inv[:, :, None]).clamp(-448.0, 448.0)
    q = torch.where(bad[:, :, None], torch.zeros_like(q), q)
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8).view(T, Kp)
    exps = torch.full((Kp // BLOCK, Tp), 127, dtype=torch.uint8, device=x.device)
    exps[:, :T] = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8).t()
    return codes, exps


def _empty_checkpoint(T, K):
    return (torch.zeros((T, _up(K, BLOCK)), dtype=torch.uint8, device="cuda"),
            torch.full((_up(K, BLOCK) // BLOCK, _up(T, BLOCK)), 127, dtype=torch.uint8, device="cuda"))


def _gate_shape(c):
    return {"channel": (c["D"],), "token": (c["T"], 1), "full": (c["T"], c["D"])}[c["gate"]]


def _norm_inputs(c, seed):
    """What both directions take: the block's output y, the residual x, the weights and the gate."""
    T, D = c["T"], c["D"]
    act, res = DTYPES[c["act"]], DTYPES[c["res"]]
    s = {"y": _activation(T, D, 0.7, seed, 0, act), "x": _activation(T, D, 2.0, seed, 2, res),
         "w_post": None, "w_pre": None, "gate": None}
    if c["post"]:
        s["w_post"] = (1.0 + _normal((D,), 0.1, seed, 4)).to(torch.bfloat16)
    if c["pre"]:
        s["w_pre"] = (1.0 + _normal((D,), 0.2, seed, 5)).to(torch.bfloat16)
    if c["gate"] != "none":
        s["gate"] = (0.5 + _normal(_gate_shape(c), 0.5, seed, 6)).to(torch.bfloat16)
    return s


def _gate_factor(gate, gate_act):
    """The factor that multiplies the block's output, in the gate's own shape."""
    if gate is None:
        return 1.0
    g = gate.to(torch.float32)
    return 1.0 / (1.0 + torch.exp(-g)) if gate_act == "sigmoid" else g


def prepare(case, seed):
    c = case
    T = c["T"]
    if c["op"] == "forward":
        D = c["D"]
        s = _norm_inputs(c, seed)
        s["r"] = torch.empty((T, D), dtype=DTYPES[c["res"]], device="cuda")
        s["h"] = torch.empty((T, D), dtype=DTYPES[c["act"]], device="cuda") if c["pre"] else None
        s["rstd_post"] = torch.empty((T,), device="cuda") if c["post"] else None
        s["rstd_pre"] = torch.empty((T,), device="cuda") if c["pre"] else None
        s["y8"] = _empty_checkpoint(T, D) if c["ckpt"] else None
        s["r8"] = _empty_checkpoint(T, D) if c["ckpt"] and c["pre"] else None
    elif c["op"] == "backward":
        D = c["D"]
        s = _norm_inputs(c, seed)
        f = _forward_plain(c, s)
        x = s.pop("x")
        y = s.pop("y")
        s["rstd_post"], s["rstd_pre"] = f["rstd_post"], f["rstd_pre"]
        s["y"] = _pack_plain(f["yh"]) if c["ckpt"] else y
        s["r"] = None if not c["pre"] else _pack_plain(f["rh"]) if c["ckpt"] else f["r"].to(DTYPES[c["res"]])
        del f, x
        s["dh"] = _normal((T, D), 1e-3, seed, 8, DTYPES[c["act"]]) if c["pre"] else None
        s["dr"] = _normal((T, D), 1e-3, seed, 9, DTYPES[c["res"]])
        s["dy"] = torch.empty((T, D), dtype=DTYPES[c["act"]], device="cuda")
        s["dx"] = torch.empty((T, D), dtype=DTYPES[c["res"]], device="cuda")
        s["dw_post"] = torch.empty((D,), device="cuda") if c["post"] else None
        s["dw_pre"] = torch.empty((D,), device="cuda") if c["pre"] else None
        s["dgate"] = None
        if c["gate"] != "none":
            s["dgate"] = torch.empty(_gate_shape(c), device="cuda",
                                     dtype=torch.bfloat16 if c["gate"] == "full" else torch.float32)
    elif c["op"] == "pack":
        s = {"x": _activation(T, c["K"], 1.0, seed, 0, DTYPES[c["dtype"]]), "out": _empty_checkpoint(T, c["K"])}
    elif c["op"] == "unpack":
        s = {"x8": _pack_plain(_activation(T, c["K"], 1.0, seed, 0, torch.float32)),
             "out": torch.empty((T, c["K"]), dtype=DTYPES[c["dtype"]], device="cuda")}
    else:
        s = {"x8": _pack_plain(_activation(T, c["K"], 1.0, seed, 0, torch.float32)),
             "dy": _normal((T, c["N"]), 1e-3, seed, 3, torch.bfloat16),
             "col": (1.0 + _normal((c["K"],), 0.2, seed, 4)).to(torch.bfloat16) if c["colscale"] else None,
             "out": torch.empty((c["N"], c["K"]), dtype=DTYPES[c["out"]], device="cuda")}
    s["case"] = dict(c)
    return s


# ---------------------------------------------------------- the plain forms --

def _forward_plain(c, s):
    y, x = s["y"].to(torch.float32), s["x"].to(torch.float32)
    f = {"rstd_post": None, "rstd_pre": None, "rh": None, "h": None}
    if c["post"]:
        f["rstd_post"] = 1.0 / torch.sqrt((y * y).mean(dim=1) + EPS)
        f["yh"] = y * f["rstd_post"][:, None]
        u = f["yh"] * s["w_post"].to(torch.float32)
    else:
        f["yh"] = u = y
    f["r"] = x + c["scale"] * _gate_factor(s["gate"], c["gate_act"]) * u
    if c["pre"]:
        f["rstd_pre"] = 1.0 / torch.sqrt((f["r"] * f["r"]).mean(dim=1) + EPS)
        f["rh"] = f["r"] * f["rstd_pre"][:, None]
        f["h"] = f["rh"] * s["w_pre"].to(torch.float32)
    return f


def _backward_plain(c, s):
    T, D = c["T"], c["D"]
    y = _values(*s["y"], T, D) if c["ckpt"] else s["y"].to(torch.float32)
    yh = y * s["rstd_post"][:, None] if c["post"] and not c["ckpt"] else y
    dr = s["dr"].to(torch.float32)
    dw_post = dw_pre = dgate = None
    if c["pre"]:
        rh = _values(*s["r"], T, D) if c["ckpt"] else s["r"].to(torch.float32) * s["rstd_pre"][:, None]
        dh = s["dh"].to(torch.float32)
        dw_pre = (dh * rh).sum(dim=0)
        wdh = dh * s["w_pre"].to(torch.float32)
        dr = dr + s["rstd_pre"][:, None] * (wdh - rh * (wdh * rh).mean(dim=1, keepdim=True))
    u = yh * s["w_post"].to(torch.float32) if c["post"] else yh
    g = _gate_factor(s["gate"], c["gate_act"])
    if c["gate"] != "none":
        dgate = c["scale"] * dr * u
        if c["gate"] == "channel":
            dgate = dgate.sum(dim=0)
        elif c["gate"] == "token":
            dgate = dgate.sum(dim=1, keepdim=True)
        if c["gate_act"] == "sigmoid":
            dgate = dgate * g * (1.0 - g)
    dy = c["scale"] * g * dr
    if c["post"]:
        dw_post = (dy * yh).sum(dim=0)
        wdy = dy * s["w_post"].to(torch.float32)
        dy = s["rstd_post"][:, None] * (wdy - yh * (wdy * yh).mean(dim=1, keepdim=True))
    return dy, dr, dw_post, dw_pre, dgate


def _checkpoint_out(pair, T, K):
    """A checkpoint's contents as the numbers they hold: e4m3 codes and power-of-two scales."""
    if pair is None:
        return None
    codes, exps = pair
    return {"codes": codes.view(torch.float8_e4m3fn)[:, :K], "scales": exps.view(torch.float8_e8m0fnu)[:, :T]}


def run(state):
    s, c = state, state["case"]
    op, T = c["op"], c["T"]
    if own:
        return _run_own(s, c, op, T)
    if op == "forward":
        f = _forward_plain(c, s)
        return {"r": f["r"].to(s["r"].dtype), "h": f["h"].to(s["h"].dtype) if c["pre"] else None,
                "rstd_post": f["rstd_post"], "rstd_pre": f["rstd_pre"],
                "y8": _checkpoint_out(_pack_plain(f["yh"]) if c["ckpt"] else None, T, c["D"]),
                "r8": _checkpoint_out(_pack_plain(f["rh"]) if c["ckpt"] and c["pre"] else None, T, c["D"])}
    if op == "backward":
        dy, dx, dw_post, dw_pre, dgate = _backward_plain(c, s)
        return {"dy": dy.to(s["dy"].dtype), "dx": dx.to(s["dx"].dtype), "dw_post": dw_post, "dw_pre": dw_pre,
                "dgate": None if dgate is None else dgate.to(s["dgate"].dtype)}
    if op == "pack":
        return _checkpoint_out(_pack_plain(s["x"].to(torch.float32)), T, c["K"])
    if op == "unpack":
        return _values(*s["x8"], T, c["K"]).to(s["out"].dtype)
    dw = s["dy"].to(torch.float32).t() @ _values(*s["x8"], T, c["K"])
    if s["col"] is not None:
        dw = dw * s["col"].to(torch.float32)
    return dw.to(s["out"].dtype)


def _run_own(s, c, op, T):
    import zero_sharded_mixed_zero1_gb300 as z
    if op in ("forward", "backward"):
        cfg = z.BlockNorm(eps=EPS, residual_scale=c["scale"], gate_act=c["gate_act"])
        D = c["D"]
    if op == "forward":
        y8 = z.Checkpoint8(T, D, *s["y8"]) if s["y8"] else None
        r8 = z.Checkpoint8(T, D, *s["r8"]) if s["r8"] else None
        z.zero1_block_norm_forward(cfg, s["y"], s["x"], s["r"], s["h"], s["rstd_post"], s["rstd_pre"],
                                   w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], y8=y8, r8=r8)
        return {"r": s["r"], "h": s["h"], "rstd_post": s["rstd_post"], "rstd_pre": s["rstd_pre"],
                "y8": _checkpoint_out(s["y8"], T, D), "r8": _checkpoint_out(s["r8"], T, D)}
    if op == "backward":
        y = z.Checkpoint8(T, D, *s["y"]) if c["ckpt"] else s["y"]
        r = z.Checkpoint8(T, D, *s["r"]) if c["ckpt"] and c["pre"] else s["r"]
        z.zero1_block_norm_backward(cfg, s["dh"], s["dr"], y, r, s["rstd_post"], s["rstd_pre"], s["dy"], s["dx"],
                                    w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], dw_post=s["dw_post"],
                                    dw_pre=s["dw_pre"], dgate=s["dgate"])
        return {"dy": s["dy"], "dx": s["dx"], "dw_post": s["dw_post"], "dw_pre": s["dw_pre"], "dgate": s["dgate"]}
    if op == "pack":
        z.zero1_checkpoint_pack(s["x"], z.Checkpoint8(T, c["K"], *s["out"]))
        return _checkpoint_out(s["out"], T, c["K"])
    if op == "unpack":
        z.zero1_checkpoint_unpack(z.Checkpoint8(T, c["K"], *s["x8"]), s["out"])
        return s["out"]
    z.zero1_weight_grad(s["dy"], z.Checkpoint8(T, c["K"], *s["x8"]), s["out"], col_scale=s["col"])
    return s["out"]


# ------------------------------------------------------------ the least work --

def work(case):
    c = case
    T = c["T"]
    if c["op"] in ("forward", "backward"):
        D = c["D"]
        a, r, n = BYTES[c["act"]], BYTES[c["res"]], T * D
        gates = {"none": 0, "channel": D, "token": T, "full": n}[c["gate"]]
        weights = D * (c["post"] + c["pre"])
        stats = 4 * T * (c["post"] + c["pre"])
        kept = n + n // BLOCK
        if c["op"] == "forward":
            b = n * (a + 2 * r + a * c["pre"]) + stats + 2 * (weights + gates) + kept * c["ckpt"] * (1 + c["pre"])
            return {"bytes": b, "flops": 12 * n}
        saved = kept * (1 + c["pre"]) if c["ckpt"] else n * (a + r * c["pre"])
        b = n * (a * (1 + c["pre"]) + 2 * r) + saved + stats + 6 * weights
        b += gates * (4 if c["gate"] == "full" else 6)
        return {"bytes": b, "flops": 30 * n}
    if c["op"] in ("pack", "unpack"):
        n = T * c["K"]
        return {"bytes": n * (BYTES[c["dtype"]] + 1) + n // BLOCK, "flops": 3 * n}
    N, K = c["N"], c["K"]
    b = 2 * T * N + T * K + T * K // BLOCK + BYTES[c["out"]] * N * K + 2 * K * c["colscale"]
    return {"bytes": b, "flops": 2 * T * N * K}


# -------------------------------------------------------------- in 64 bits --

def _exact_values(codes, exps, T, K):
    """Sign, exponent and mantissa fields of the codes by the format's definition, in float64."""
    b = codes.to(torch.int64)
    field, frac = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(field == 0, frac * 2.0 ** -9, torch.ldexp(1.0 + frac / 8.0, field - 7))
    mag = torch.where(b >= 128, -mag, mag)
    e = exps[:, :T].to(torch.int64).t() - 127
    Kp = codes.shape[1]
    return torch.ldexp(mag.view(T, Kp // BLOCK, BLOCK), e[:, :, None]).view(T, Kp)[:, :K]


def _exact_pack(x):
    """Scales by search over exponents' definition and codes by rounding to the grid, half to even."""
    T, K = x.shape
    Kp = _up(K, BLOCK)
    v = torch.nn.functional.pad(x, (0, Kp - K)).view(T, Kp // BLOCK, BLOCK)
    amax = v.abs().amax(dim=2)
    e = torch.ceil(torch.log2((amax / 448.0).clamp_min(2.0 ** -119))).clamp(-119, 119)
    e = torch.where(torch.ldexp(torch.full_like(e, 448.0), e) < amax, e + 1, e)        # log2's own rounding
    e = torch.where((torch.ldexp(torch.full_like(e, 224.0), e) >= amax) & (e > -119), e - 1, e)
    q = torch.ldexp(v, -e[:, :, None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3.0)
    q = torch.round(q / step) * step
    return {"codes": q.view(T, Kp)[:, :K], "scales": torch.exp2(e).t()}


def exact(case, seed):
    c, s = case, prepare(case, seed)
    T = c["T"]
    if c["op"] == "pack":
        return _exact_pack(s["x"].double())
    if c["op"] == "unpack":
        return _exact_values(*s["x8"], T, c["K"])
    if c["op"] == "weight_grad":
        x = _exact_values(*s["x8"], T, c["K"])
        if s["col"] is not None:
            x = x * s["col"].double()
        return torch.einsum("tn,tk->nk", s["dy"].double(), x)
    D = c["D"]
    up = lambda t: None if t is None else t.double()  # noqa: E731
    w_post, w_pre, gate = up(s["w_post"]), up(s["w_pre"]), up(s["gate"])
    g = torch.ones((), dtype=torch.float64, device="cuda") if gate is None else \
        torch.sigmoid(gate) if c["gate_act"] == "sigmoid" else gate
    if c["op"] == "forward":
        y = up(s["y"])
        out = {"rstd_post": None, "rstd_pre": None, "h": None, "y8": None, "r8": None}
        yh, u = y, y
        if c["post"]:
            out["rstd_post"] = (y.square().sum(1) / D + EPS).rsqrt()
            yh = y * out["rstd_post"].unsqueeze(1)
            u = yh * w_post
        del y
        if c["ckpt"]:
            out["y8"] = _exact_pack(yh)
        out["r"] = up(s["x"]).addcmul_(u * g, torch.full((), c["scale"], dtype=torch.float64, device="cuda"))
        if c["pre"]:
            out["rstd_pre"] = (out["r"].square().sum(1) / D + EPS).rsqrt()
            rh = out["r"] * out["rstd_pre"].unsqueeze(1)
            out["h"] = rh * w_pre
            if c["ckpt"]:
                out["r8"] = _exact_pack(rh)
        return out
    out = {"dw_post": None, "dw_pre": None, "dgate": None}
    r1, r2 = up(s["rstd_post"]), up(s["rstd_pre"])
    dx = up(s["dr"])
    if c["pre"]:
        rh = _exact_values(*s["r"], T, D) if c["ckpt"] else up(s["r"]) * r2.unsqueeze(1)
        dh = up(s["dh"])
        out["dw_pre"] = torch.einsum("td,td->d", dh, rh)
        dh *= w_pre
        dx = dx + (dh - rh * (torch.einsum("td,td->t", dh, rh) / D).unsqueeze(1)) * r2.unsqueeze(1)
        del dh, rh
    yh = _exact_values(*s["y"], T, D) if c["ckpt"] else up(s["y"]) * (r1.unsqueeze(1) if c["post"] else 1.0)
    if gate is not None:
        u = yh * (w_post if c["post"] else 1.0) * c["scale"]
        slope = g * (1.0 - g) if c["gate_act"] == "sigmoid" else torch.ones_like(g)
        if c["gate"] == "channel":
            out["dgate"] = torch.einsum("td,td->d", dx, u) * slope
        elif c["gate"] == "token":
            out["dgate"] = torch.einsum("td,td->t", dx, u).unsqueeze(1) * slope
        else:
            out["dgate"] = dx * u * slope
        del u
    dyh = dx * g * c["scale"]
    if c["post"]:
        out["dw_post"] = torch.einsum("td,td->d", dyh, yh)
        dyh = dyh * w_post
        dyh = (dyh - yh * (torch.einsum("td,td->t", dyh, yh) / D).unsqueeze(1)) * r1.unsqueeze(1)
    out["dx"], out["dy"] = dx, dyh
    return out
