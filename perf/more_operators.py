"""The operators of a training block and of its step, second set, as they are
measured: the global gradient norm with clipping (over many tensors, and in
the sharded step), layer norm with its residual (forward, backward), and the
gated feed-forward block (forward, backward with the pre-activations computed
again, and the gradients of its input and weights).

A checkpoint of a [T, D] activation is a pair of uint8 tensors: `codes`
[T, Dp] (e4m3, Dp = D rounded up to 128) and `exps` [Dp / 128, Tp] (Tp = T
rounded up to 128): exps[b, t] = e + 127 is the power-of-two scale of row t's
columns [128 b, 128 b + 128), so a value is code * 2^e; 255 marks a block that
stands for NaN.  e is the smallest exponent in [-119, 119] with
max|x| <= 448 * 2^e.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-5          # of layer norm
CLIP_EPS = 1e-6     # added to the norm that divides
BLOCK = 128
ADAMW = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1}
BATCH, STEP = 1024, 10
GELU_A, GELU_B = math.sqrt(2.0 / math.pi), 0.044715


def _up(n, m):
    return -(-n // m) * m


# ---------------------------------------------------------------- the cases --

def _clip(count, numel, layers, dtype, ratio):
    """`ratio`: the largest norm allowed, as a multiple of the norm that is expected."""
    return {"op": "clip", "count": count, "numel": numel, "layers": layers, "dtype": dtype, "ratio": ratio}


def _step(n, M, align, ratio, kept):
    return {"op": "step", "n": n, "M": M, "align": align, "ratio": ratio, "kept": kept}


def _ln(op, T, D, act, res, params, residual, ckpt, grads="f32"):
    return {"op": op, "T": T, "D": D, "act": act, "res": res, "params": params, "residual": residual, "ckpt": ckpt,
            "grads": grads}


def _ffn(op, T, D, F, act="silu", grads="bf16"):
    return {"op": op, "T": T, "D": D, "F": F, "act": act, "grads": grads}


def listed():
    named = [
        # a handful of small parameters, of odd sizes and at odd places of a flat buffer: launch latency
        ("clip_few_small", _clip(24, 50000, 0, "bf16", 0.5)),
        # the gradients of four Llama-style layers, 36 tensors of one flat buffer, each with its own norm
        ("clip_llama_layers", _clip(36, 872448000, 4, "bf16", 0.3)),
        # the smallest optimizer step, whose gradients are below the largest norm: nothing is scaled
        ("step_tiny_1M_M4", _step(1048576, 4, 128, 2.0, False)),
        # the GPT-2-small-sized step over eight replicas, clipped, the sums kept between the two passes
        ("step_gpt2_small_124M_M8", _step(124439808, 8, 1, 0.25, True)),
        # a micro-batch at the Llama layers' width: the residual stream and its norm, with a checkpoint
        ("layer_norm_forward_block", _ln("ln_forward", 8192, 4096, "bf16", "bf16", "bf16", True, True)),
        # an odd width, fp32 throughout, no residual: a small model's head
        ("layer_norm_backward_odd_f32", _ln("ln_backward", 2003, 1021, "f32", "f32", "f32", False, False)),
        # the backward pass of layer_norm_forward_block from its checkpoint
        ("layer_norm_backward_block", _ln("ln_backward", 8192, 4096, "bf16", "bf16", "bf16", True, True)),
        # a few tokens through a small model's block: latency
        ("ffn_forward_short", _ffn("ffn_forward", 16, 768, 2048, "gelu")),
        # a micro-batch through the feed-forward block of the Llama layers
        ("ffn_forward_block", _ffn("ffn_forward", 8192, 4096, 14336)),
        # its backward pass up to the gradients of the pre-activations
        ("ffn_backward_block", _ffn("ffn_backward", 8192, 4096, 14336)),
        # the gradients of its input and of both weights
        ("ffn_grads_block", _ffn("ffn_grads", 8192, 4096, 14336)),
        # the same at odd sizes, with fp32 weight gradients
        ("ffn_grads_odd_f32", _ffn("ffn_grads", 777, 1000, 1371, "silu", "f32")),
    ]
    return [dict(c, name=n) for n, c in named]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi):
    """A size of [lo, hi]: half of them multiples of 64 as models have them, half anything."""
    n = _log_int(rng, lo, hi)
    return max(lo, min(hi, _up(n, 64))) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(["clip", "step", "ln_forward", "ln_backward", "ffn_forward", "ffn_backward", "ffn_grads", "ffn_grads"])
    if op == "clip":
        return _clip(rng.randint(1, 48), _log_int(rng, 1000, 1 << 28), 0, rng.choice(["bf16", "bf16", "f32"]),
                     rng.choice([0.1, 0.5, 1.5]))
    if op == "step":
        M = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
        return _step(_log_int(rng, 1000, (1 << 29) // max(M, 4)), M, rng.choice([1, 8, 128]), rng.choice([0.1, 0.5, 1.5]),
                     rng.random() < 0.5)
    if op in ("ln_forward", "ln_backward"):
        D = _size(rng, 64, 16384)
        T = _log_int(rng, 1, min(32768, (1 << 25) // D))
        act, res = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        return _ln(op, T, D, act, res, rng.choice(["bf16", "f32"]), rng.random() < 0.6, rng.random() < 0.4,
                   rng.choice(["bf16", "f32"]))
    D, F = _size(rng, 64, 8192), _size(rng, 64, 16384)
    T = _log_int(rng, 1, min(16384, 8192 * 4096 * 14336 // (D * F)))
    return _ffn(op, T, D, F, rng.choice(["silu", "gelu"]), rng.choice(["bf16", "bf16", "f32"]))


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


def _tensor_sizes(c):
    """The sizes of a clip case's tensors: those of Llama-style layers, or cuts at random places."""
    if c["layers"]:
        d, kv, f = 4096, 1024, 14336
        return [d * d, kv * d, kv * d, d * d, f * d, f * d, d * f, d, d] * c["layers"]
    cuts = random.Random(c["count"] * 1000003 + c["numel"])
    at = sorted(cuts.randint(0, c["numel"]) for _ in range(c["count"] - 1))
    return [b - a for a, b in zip([0] + at, at + [c["numel"]])]


def _views(flat, sizes):
    return list(torch.split(flat, sizes))


def _values(codes, exps, T, D):
    """The fp32 values that a checkpoint stands for."""
    e = exps[:, :T]
    s = (e.to(torch.int32) << 23).view(torch.float32)
    s = torch.where(e == 255, torch.full_like(s, float("nan")), s).t().repeat_interleave(BLOCK, dim=1)
    return (codes.view(torch.float8_e4m3fn).float() * s)[:, :D].contiguous()


def _pack_plain(x):
    """codes, exps of an fp32 [T, D] tensor."""
    T, D = x.shape
    Dp, Tp = _up(D, BLOCK), _up(T, BLOCK)
    v = torch.zeros((T, Dp), device=x.device)
    v[:, :D] = x
    v = v.view(T, Dp // BLOCK, BLOCK)
    amax = v.abs().amax(dim=2)
    bad = ~torch.isfinite(amax)
    m, e = torch.frexp(torch.where(bad, torch.zeros_like(amax), amax))  # amax = m 2^e, 0.5 <= m < 1
    e = (e - 9 + (m > 0.875).int()).clamp(-119, 119)                    # 448 = 0.875 * 2^9
    inv = ((127 - e) << 23).view(torch.float32)
    q = (v * inv[:, :, None]).clamp(-448.0, 448.0)
    q = torch.where(bad[:, :, None], torch.zeros_like(q), q)
    codes = q.to(torch.float8_e4m3fn).view(torch.uint8).view(T, Dp)
    exps = torch.full((Dp // BLOCK, Tp), 127, dtype=torch.uint8, device=x.device)
    exps[:, :T] = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8).t()
    return codes, exps


def _empty_checkpoint(T, D):
    return (torch.zeros((T, _up(D, BLOCK)), dtype=torch.uint8, device="cuda"),
            torch.full((_up(D, BLOCK) // BLOCK, _up(T, BLOCK)), 127, dtype=torch.uint8, device="cuda"))


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    c = case
    s = {"case": dict(c)}
    if c["op"] == "clip":
        # gradients of many tensors in one flat buffer; every tensor with a size of its own
        dt = DTYPES[c["dtype"]]
        s["grads"] = _views(_normal((c["numel"],), 1e-3, seed, 0, dt), _tensor_sizes(c))
        s["outs"] = _views(_empty((c["numel"],), dt), _tensor_sizes(c))
        s["max_norm"] = c["ratio"] * 1e-3 * math.sqrt(c["numel"])
        s["sumsq"], s["norms"] = _empty((1,), torch.float64), _empty((c["count"],), torch.float32)
        s["norm"] = _empty((1,), torch.float32)
    elif c["op"] == "step":
        n, M = c["n"], c["M"]
        P = _up(n, M * c["align"])
        # a replica's gradient is a sum over its samples
        s["grads"] = [_normal((n,), 1e-2, seed, r, torch.bfloat16) for r in range(M)]
        s["max_norm"] = c["ratio"] * 1e-2 * math.sqrt(float(n) * M) / BATCH
        s["master"], s["m"] = torch.zeros(P, device="cuda"), torch.zeros(P, device="cuda")
        s["v"] = torch.zeros(P, device="cuda")
        s["master"][:n] = _normal((n,), 0.02, seed, 60)
        s["m"][:n] = _normal((n,), 1e-5, seed, 61)
        s["v"][:n] = _normal((n,), 1e-5, seed, 62).square_()
        s["out"] = [torch.empty_like(s[k]) for k in ("master", "m", "v")]
        s["params"] = _empty((n,), torch.bfloat16)
        s["sums"] = _empty((P,), torch.float32) if c["kept"] else None
        s["sumsq"], s["norm"] = _empty((1,), torch.float64), _empty((1,), torch.float32)
    elif c["op"] in ("ln_forward", "ln_backward"):
        T, D = c["T"], c["D"]
        act, res = DTYPES[c["act"]], DTYPES[c["res"]]
        s["scale"] = 0.5 if c["residual"] else 1.0
        s["w"] = (1.0 + _normal((D,), 0.2, seed, 4)).to(DTYPES[c["params"]])
        s["b"] = _normal((D,), 0.2, seed, 5, DTYPES[c["params"]])
        x = _activation(T, D, 2.0, seed, 0, res)
        x += _normal((D,), 0.5, seed, 6, res)  # channels have means of their own
        y = _activation(T, D, 0.7, seed, 2, act) if c["residual"] else None
        if c["op"] == "ln_forward":
            s["x"], s["y"] = x, y
            s["r"] = _empty((T, D), res) if c["residual"] else None
            s["h"] = _empty((T, D), act)
            s["mean"], s["rstd"] = _empty((T,), torch.float32), _empty((T,), torch.float32)
            s["r8"] = _empty_checkpoint(T, D) if c["ckpt"] else None
        else:
            f = _ln_forward_plain({**s, "x": x, "y": y}, c)
            s["mean"], s["rstd"] = f["mean"], f["rstd"]
            s["r"] = _pack_plain(f["rh"]) if c["ckpt"] else f["r"].to(res)
            del f, x, y
            s["dh"] = _normal((T, D), 1e-3, seed, 8, act)
            s["dr"] = _normal((T, D), 1e-3, seed, 9, res) if c["residual"] else None
            s["dx"] = _empty((T, D), res)
            s["dy"] = _empty((T, D), act) if c["residual"] else None
            s["dw"], s["db"] = _empty((D,), DTYPES[c["grads"]]), _empty((D,), DTYPES[c["grads"]])
    else:
        T, D, F = c["T"], c["D"], c["F"]
        bf = torch.bfloat16
        s["h"] = _normal((T, D), 1.0, seed, 0, bf)
        if c["op"] != "ffn_grads":
            s["w_gate"], s["w_up"] = _normal((F, D), D ** -0.5, seed, 2, bf), _normal((F, D), D ** -0.5, seed, 3, bf)
            s["a"] = _empty((T, F), bf)
        else:
            s["w_gate"], s["w_up"] = _normal((F, D), 0.02, seed, 2, bf), _normal((F, D), 0.02, seed, 3, bf)
        if c["op"] == "ffn_backward":
            s["da"] = _normal((T, F), 1e-3, seed, 4, bf)
            s["dg"], s["du"] = _empty((T, F), bf), _empty((T, F), bf)
        if c["op"] == "ffn_grads":
            s["dg"], s["du"] = _normal((T, F), 1e-3, seed, 4, bf), _normal((T, F), 1e-3, seed, 5, bf)
            s["dh"] = _empty((T, D), bf)
            s["dw_gate"], s["dw_up"] = _empty((F, D), DTYPES[c["grads"]]), _empty((F, D), DTYPES[c["grads"]])
    return s


# ---------------------------------------------------------- the plain forms --

def _coef(norm, max_norm):
    return (max_norm / (norm + CLIP_EPS)).clamp(max=1.0)


def _clip_plain(s, c):
    sumsq = torch.stack([g.double().square().sum() for g in s["grads"]])
    norm = sumsq.sum().sqrt()
    coef = _coef(norm, s["max_norm"]).float()
    return {"norm": norm.float().view(1), "norms": sumsq.sqrt().float(),
            "grads": [(g.float() * coef).to(g.dtype) for g in s["grads"]]}


def _step_plain(s, c):
    n, h = c["n"], ADAMW
    g = s["grads"][0].float()
    for r in s["grads"][1:]:
        g = g + r.float()
    g = g * (1.0 / BATCH)
    norm = g.double().square().sum().sqrt()
    full = torch.zeros_like(s["master"])
    full[:n] = g * _coef(norm, s["max_norm"]).float()
    m = h["beta1"] * s["m"] + (1.0 - h["beta1"]) * full
    v = h["beta2"] * s["v"] + (1.0 - h["beta2"]) * (full * full)
    u = (m / (1.0 - h["beta1"] ** STEP)) / (torch.sqrt(v / (1.0 - h["beta2"] ** STEP)) + h["eps"])
    w = s["master"] * (1.0 - h["lr"] * h["weight_decay"]) - h["lr"] * u
    return {"norm": norm.float().view(1), "master": w, "m": m, "v": v, "params": w[:n].to(torch.bfloat16)}


def _ln_forward_plain(s, c):
    r = s["x"].float()
    if s["y"] is not None:
        r = r + s["scale"] * s["y"].float()
    mean = r.mean(dim=1)
    d = r - mean[:, None]
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1) + EPS)
    rh = d * rstd[:, None]
    return {"r": r, "mean": mean, "rstd": rstd, "rh": rh, "h": rh * s["w"].float() + s["b"].float()}


def _ln_backward_plain(s, c):
    if c["ckpt"]:
        rh = _values(*s["r"], c["T"], c["D"])
    else:
        rh = (s["r"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dh = s["dh"].float()
    t = dh * s["w"].float()
    d = s["rstd"][:, None] * (t - t.mean(dim=1, keepdim=True) - rh * (t * rh).mean(dim=1, keepdim=True))
    if s["dr"] is not None:
        d = d + s["dr"].float()
    return {"dx": d.to(s["dx"].dtype), "dy": None if s["dy"] is None else (s["scale"] * d).to(s["dy"].dtype),
            "dw": (dh * rh).sum(dim=0).to(s["dw"].dtype), "db": dh.sum(dim=0).to(s["db"].dtype)}


def _act_plain(g, act):
    """act(g) = g s(k(g)) and its derivative; s the logistic function, k(g) = g (silu) or that of gelu's tanh form."""
    if act == "silu":
        k, dk = g, 1.0
    else:
        k, dk = 2.0 * GELU_A * (g + GELU_B * g * g * g), 2.0 * GELU_A * (1.0 + 3.0 * GELU_B * g * g)
    s = 1.0 / (1.0 + torch.exp(-k))
    return g * s, s + g * s * (1.0 - s) * dk


def _ffn_forward_plain(s, c):
    h = s["h"].float()
    g, u = h @ s["w_gate"].float().t(), h @ s["w_up"].float().t()
    return (_act_plain(g, c["act"])[0] * u).to(torch.bfloat16)


def _ffn_backward_plain(s, c):
    h, da = s["h"].float(), s["da"].float()
    g, u = h @ s["w_gate"].float().t(), h @ s["w_up"].float().t()
    f, df = _act_plain(g, c["act"])
    return {"a": (f * u).to(torch.bfloat16), "dg": (da * u * df).to(torch.bfloat16), "du": (da * f).to(torch.bfloat16)}


def _ffn_grads_plain(s, c):
    dg, du, h = s["dg"].float(), s["du"].float(), s["h"].float()
    return {"dh": (dg @ s["w_gate"].float() + du @ s["w_up"].float()).to(torch.bfloat16),
            "dw_gate": (dg.t() @ h).to(s["dw_gate"].dtype), "dw_up": (du.t() @ h).to(s["dw_up"].dtype)}


def _checkpoint_out(pair, T, D):
    """A checkpoint's contents as the numbers they hold: e4m3 codes and power-of-two scales."""
    if pair is None:
        return None
    codes, exps = pair
    return {"codes": codes.view(torch.float8_e4m3fn)[:, :D], "scales": exps.view(torch.float8_e8m0fnu)[:, :T]}


def run(state):
    s, c = state, state["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "clip":
        return _clip_plain(s, c)
    if c["op"] == "step":
        return _step_plain(s, c)
    if c["op"] == "ln_forward":
        f = _ln_forward_plain(s, c)
        return {"r": None if s["r"] is None else f["r"].to(s["r"].dtype), "h": f["h"].to(s["h"].dtype),
                "mean": f["mean"], "rstd": f["rstd"],
                "r8": _checkpoint_out(_pack_plain(f["rh"]) if c["ckpt"] else None, c["T"], c["D"])}
    if c["op"] == "ln_backward":
        return _ln_backward_plain(s, c)
    if c["op"] == "ffn_forward":
        return _ffn_forward_plain(s, c)
    if c["op"] == "ffn_backward":
        return _ffn_backward_plain(s, c)
    return _ffn_grads_plain(s, c)


def _run_own(s, c):
    import zero_sharded_mixed_zero1_gb300 as z
    if c["op"] == "clip":
        z.zero1_grad_sumsq(s["grads"], s["sumsq"], norms=s["norms"])
        z.zero1_grad_clip(s["grads"], s["sumsq"], s["max_norm"], outs=s["outs"], norm=s["norm"])
        return {"norm": s["norm"], "norms": s["norms"], "grads": s["outs"]}
    if c["op"] == "step":
        plan = z.zero1_plan(c["n"], c["M"], c["align"])
        hp = z.AdamW(global_batch=BATCH, step=STEP, **ADAMW)
        z.zero1_shard_grad_sumsq(plan, 0, c["M"], s["grads"], hp, s["sumsq"], sums=s["sums"])
        z.zero1_step_clipped(plan, 0, c["M"], s["grads"], s["master"], s["m"], s["v"], s["params"], hp, s["sumsq"],
                             s["max_norm"], sums=s["sums"], out=s["out"], norm=s["norm"])
        return {"norm": s["norm"], "master": s["out"][0], "m": s["out"][1], "v": s["out"][2], "params": s["params"]}
    T, D = c["T"], c["D"]
    if c["op"] == "ln_forward":
        r8 = z.Checkpoint8(T, D, *s["r8"]) if c["ckpt"] else None
        z.zero1_layer_norm_forward(z.LayerNorm(eps=EPS, residual_scale=s["scale"]), s["x"], s["h"], s["mean"], s["rstd"],
                                   w=s["w"], b=s["b"], y=s["y"], r=s["r"], r8=r8)
        return {"r": s["r"], "h": s["h"], "mean": s["mean"], "rstd": s["rstd"], "r8": _checkpoint_out(s["r8"], T, D)}
    if c["op"] == "ln_backward":
        r = z.Checkpoint8(T, D, *s["r"]) if c["ckpt"] else s["r"]
        z.zero1_layer_norm_backward(z.LayerNorm(eps=EPS, residual_scale=s["scale"]), s["dh"], s["dr"], r, s["mean"],
                                    s["rstd"], s["dx"], dy=s["dy"], w=s["w"], dw=s["dw"], db=s["db"])
        return {"dx": s["dx"], "dy": s["dy"], "dw": s["dw"], "db": s["db"]}
    if c["op"] == "ffn_forward":
        z.zero1_gated_ffn_forward(s["h"], s["w_gate"], s["w_up"], s["a"], act=c["act"])
        return s["a"]
    if c["op"] == "ffn_backward":
        z.zero1_gated_ffn_backward(s["da"], s["h"], s["w_gate"], s["w_up"], s["dg"], s["du"], a=s["a"], act=c["act"])
        return {"a": s["a"], "dg": s["dg"], "du": s["du"]}
    z.zero1_gated_ffn_input_grad(s["dg"], s["du"], s["w_gate"], s["w_up"], s["dh"])
    z.zero1_weight_grad_bf16(s["dg"], s["h"], s["dw_gate"])
    z.zero1_weight_grad_bf16(s["du"], s["h"], s["dw_up"])
    return {"dh": s["dh"], "dw_gate": s["dw_gate"], "dw_up": s["dw_up"]}


# ------------------------------------------------------------ the least work --

def work(case):
    c = case
    if c["op"] == "clip":
        return {"bytes": 2 * c["numel"] * BYTES[c["dtype"]], "flops": 3 * c["numel"]}
    if c["op"] == "step":
        # gradients once, the state read and written, the parameters written
        return {"bytes": c["n"] * (2 * c["M"] + 26), "flops": c["n"] * (c["M"] + 20)}
    T, D = c["T"], c["D"]
    if c["op"] in ("ln_forward", "ln_backward"):
        a, r, n, p = BYTES[c["act"]], BYTES[c["res"]], T * D, BYTES[c["params"]]
        kept = n + n // BLOCK
        if c["op"] == "ln_forward":
            b = n * (a + r + (a + r) * c["residual"]) + kept * c["ckpt"] + 8 * T + 2 * p * D
            return {"bytes": b, "flops": 10 * n}
        b = n * (a + r + (a + r) * c["residual"]) + (kept if c["ckpt"] else n * r) + 8 * T + D * (p + 2 * BYTES[c["grads"]])
        return {"bytes": b, "flops": 15 * n}
    F = c["F"]
    if c["op"] == "ffn_forward":
        return {"bytes": 2 * (T * D + 2 * F * D + T * F), "flops": 4 * T * D * F}
    if c["op"] == "ffn_backward":
        return {"bytes": 2 * (T * D + 2 * F * D + 4 * T * F), "flops": 4 * T * D * F}
    return {"bytes": 2 * (2 * T * F + 2 * T * D + 2 * F * D) + 2 * BYTES[c["grads"]] * F * D, "flops": 8 * T * D * F}


# -------------------------------------------------------------- in 64 bits --

def _exact_values(codes, exps, T, D):
    """Sign, exponent and mantissa fields of the codes by the format's definition, in float64."""
    b = codes.to(torch.int64)
    field, frac = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(field == 0, frac * 2.0 ** -9, torch.ldexp(1.0 + frac / 8.0, field - 7))
    mag = torch.where(b >= 128, -mag, mag)
    e = exps[:, :T].to(torch.int64).t() - 127
    Dp = codes.shape[1]
    return torch.ldexp(mag.view(T, Dp // BLOCK, BLOCK), e[:, :, None]).view(T, Dp)[:, :D]


def _exact_pack(x):
    """Scales by search over exponents' definition and codes by rounding to the grid, half to even."""
    T, D = x.shape
    Dp = _up(D, BLOCK)
    v = torch.nn.functional.pad(x, (0, Dp - D)).view(T, Dp // BLOCK, BLOCK)
    amax = v.abs().amax(dim=2)
    e = torch.ceil(torch.log2((amax / 448.0).clamp_min(2.0 ** -119))).clamp(-119, 119)
    e = torch.where(torch.ldexp(torch.full_like(e, 448.0), e) < amax, e + 1, e)        # log2's own rounding
    e = torch.where((torch.ldexp(torch.full_like(e, 224.0), e) >= amax) & (e > -119), e - 1, e)
    q = torch.ldexp(v, -e[:, :, None]).clamp(-448.0, 448.0)
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -6))) - 3.0)
    q = torch.round(q / step) * step
    return {"codes": q.view(T, Dp)[:, :D], "scales": torch.exp2(e).t()}


def _exact_gate(g, act):
    """(act(g), act'(g)): silu by the logistic function, gelu by its tanh form."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1.0 + g * torch.sigmoid(-g))
    t = torch.tanh(GELU_A * (g + GELU_B * g.pow(3)))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * GELU_A * (1.0 + 3.0 * GELU_B * g * g)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "clip":
        norms = torch.stack([torch.linalg.vector_norm(g, dtype=f64) for g in s["grads"]])
        norm = torch.linalg.vector_norm(norms)
        k = min(1.0, s["max_norm"] / (norm.item() + CLIP_EPS))
        return {"norm": norm.view(1), "norms": norms, "grads": [g.to(f64).mul_(k) for g in s["grads"]]}
    if c["op"] == "step":
        n, h = c["n"], ADAMW
        g = torch.zeros(s["master"].numel(), dtype=f64, device="cuda")
        for r in s["grads"]:
            g[:n] += r
        g /= BATCH
        norm = torch.linalg.vector_norm(g)
        g *= min(1.0, s["max_norm"] / (norm.item() + CLIP_EPS))
        m = s["m"].to(f64).mul_(h["beta1"]).add_(g, alpha=1.0 - h["beta1"])
        v = s["v"].to(f64).mul_(h["beta2"]).addcmul_(g, g, value=1.0 - h["beta2"])
        del g
        den = v.div(1.0 - h["beta2"] ** STEP).sqrt_().add_(h["eps"])
        w = s["master"].to(f64).mul_(1.0 - h["lr"] * h["weight_decay"])
        w.addcdiv_(m, den, value=-h["lr"] / (1.0 - h["beta1"] ** STEP))
        return {"norm": norm.view(1), "master": w, "m": m, "v": v, "params": w[:n]}
    up = lambda t: None if t is None else t.to(f64)  # noqa: E731
    T, D = c["T"], c["D"]
    if c["op"] == "ln_forward":
        r = up(s["x"])
        if s["y"] is not None:
            r = r.add_(up(s["y"]), alpha=s["scale"])
        var, mean = torch.var_mean(r, dim=1, correction=0)
        rstd = (var + EPS).rsqrt()
        rh = (r - mean.unsqueeze(1)).mul_(rstd.unsqueeze(1))
        return {"r": None if s["r"] is None else r, "mean": mean, "rstd": rstd,
                "r8": _exact_pack(rh) if c["ckpt"] else None,
                "h": torch.addcmul(up(s["b"]), rh, up(s["w"]))}
    if c["op"] == "ln_backward":
        rstd = up(s["rstd"]).unsqueeze(1)
        rh = _exact_values(*s["r"], T, D) if c["ckpt"] else (up(s["r"]) - up(s["mean"]).unsqueeze(1)) * rstd
        dh = up(s["dh"])
        out = {"dw": torch.einsum("td,td->d", dh, rh), "db": dh.sum(0), "dy": None}
        t = dh * up(s["w"])
        rows = torch.stack([t.sum(1), torch.einsum("td,td->t", t, rh)], 1) / D
        d = (t - rows[:, :1] - rh * rows[:, 1:]) * rstd
        if s["dr"] is not None:
            d = d + up(s["dr"])
        out["dx"] = d
        if s["dy"] is not None:
            out["dy"] = d * s["scale"]
        return out
    if c["op"] == "ffn_grads":
        dg, du, h = up(s["dg"]), up(s["du"]), up(s["h"])
        dh = torch.mm(dg, up(s["w_gate"]))
        return {"dh": dh.addmm_(du, up(s["w_up"])), "dw_gate": torch.einsum("tf,td->fd", dg, h),
                "dw_up": torch.einsum("tf,td->fd", du, h)}
    h = up(s["h"])
    g, u = torch.einsum("td,fd->tf", h, up(s["w_gate"])), torch.einsum("td,fd->tf", h, up(s["w_up"]))
    f, df = _exact_gate(g, c["act"])
    if c["op"] == "ffn_forward":
        return f.mul_(u)
    da = up(s["da"])
    return {"a": f * u, "dg": df.mul_(u).mul_(da), "du": f.mul_(da)}
