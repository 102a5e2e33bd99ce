"""Block norms with gate and residual scale, 8-bit activation checkpoints and
the weight gradient from a checkpoint, against the 64-bit formulas of
block_reference.py, within bounds derived there."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
import block_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rand(shape, std, seed, dtype=F32):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F32) * std).to(dtype)


def dev(t, cuda, pad=0, off=0):
    """On the GPU; pad > 0 makes the rows strided, off shifts the base."""
    if t is None:
        return None
    if t.dim() == 1:
        big = torch.full((t.shape[0] + off,), 7.0, dtype=t.dtype, device=cuda)
        big[off:] = t.to(cuda)
        return big[off:]
    T, D = t.shape
    big = torch.full((T * (D + pad) + off,), 7.0, dtype=t.dtype, device=cuda)
    v = big[off:].view(T, D + pad)[:, :D]
    v.copy_(t)
    return v


def empty(T, D, dtype, cuda, pad=0, off=0):
    return dev(torch.full((T, D), float("nan"), dtype=dtype), cuda, pad, off)


def check(got, want, bound, what):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, what
    err = (got - want).abs()
    bad = ~(err <= bound + ref.TINY)
    if bad.any():
        j = bad.flatten().nonzero()[0].item()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {j}: "
                             f"{got.flatten()[j].item()} vs {want.flatten()[j].item()}, "
                             f"bound {(bound + torch.zeros_like(err)).flatten()[j].item():.3g}")


def fill_checkpoint(k, x64):
    codes, exps = ref.pack(x64)
    k.codes.copy_(codes)
    k.exps[:, :k.rows].copy_(exps.t())


def checkpoint_values(k):
    return ref.values(k.codes.cpu(), k.exps[:, :k.rows].t().cpu(), k.cols)


# ------------------------------------------------------------- checkpoints ---

PACK_SHAPES = [(1, 1), (1, 128), (2, 127), (3, 129), (5, 8), (4, 256), (7, 1000), (33, 640), (130, 2056), (1, 16385),
               (257, 136)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,K", PACK_SHAPES)
@pytest.mark.parametrize("pad,off", [(0, 0), (8, 0), (3, 1)])
def test_pack_and_unpack_are_exact(cuda_device, dtype, T, K, pad, off):
    x = rand((T, K), 1.0, T * 7 + K)
    x *= torch.exp(rand((T, 1), 6.0, 3))        # rows over many binades
    x[0, ::3] = 0.0
    x[-1, K // 2] *= 300.0                      # an outlier in a block
    x = x.to(dtype)
    k = z.new_checkpoint(T, K, cuda_device)
    k.codes.fill_(0x55)
    k.exps.fill_(0xAA)
    z.zero1_checkpoint_pack(dev(x, cuda_device, pad, off), k)
    codes, exps = ref.pack(x.double())
    assert torch.equal(k.codes.cpu(), codes)
    assert torch.equal(k.exps[:, :T].cpu(), exps.t())
    assert (k.exps[:, T:] == 0xAA).all()        # nothing written past the rows
    want = ref.values(codes, exps, K)
    for out_dtype in (BF16, F32):
        out = empty(T, K, out_dtype, cuda_device, pad, off)
        z.zero1_checkpoint_unpack(k, out)
        assert torch.equal(out.double().cpu(), want)


def test_pack_rounds_every_code_and_tie_as_defined(cuda_device):
    grid = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (grid[1:] + grid[:-1]) / 2                                # ties
    x = torch.cat([grid, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    x = torch.cat([x, -x])
    rows = torch.zeros((x.numel(), 128))
    rows[:, 0] = 448.0                                              # fixes the scale at 1
    rows[:, 5] = x
    k = z.new_checkpoint(rows.shape[0], 128, cuda_device)
    z.zero1_checkpoint_pack(rows.to(cuda_device), k)
    codes, exps = ref.pack(rows.double())
    assert torch.equal(k.codes.cpu(), codes)
    assert (exps == 127).all() and torch.equal(k.exps[0, :rows.shape[0]].cpu(), exps[:, 0])


@pytest.mark.parametrize("amax", [448.0, 448.0000305, 464.0, 1.75, 1.7500001, 1e-30, 2.0 ** -119 * 448, 2.0 ** -126,
                                  1e-40, 2.0 ** 119 * 448, 3.4e38, 0.0])
def test_pack_scale_boundaries(cuda_device, amax):
    x = torch.zeros((2, 200))
    x[0, 130] = amax
    x[1, 3] = -amax
    x[1, 4] = amax / 3
    k = z.new_checkpoint(2, 200, cuda_device)
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    codes, exps = ref.pack(x.double())
    assert torch.equal(k.codes.cpu(), codes) and torch.equal(k.exps[:, :2].cpu(), exps.t())
    out = torch.empty((2, 200), device=cuda_device)
    z.zero1_checkpoint_unpack(k, out)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype,K", [(BF16, 384), (F32, 300)])
def test_block_with_a_non_finite_value_stands_for_nan(cuda_device, bad, dtype, K):
    x = rand((3, K), 1.0, 5, dtype)
    x[1, 200] = bad
    k = z.new_checkpoint(3, K, cuda_device)
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    assert k.exps[1, 1] == 255 and (k.codes[1, 128:256] == 0).all()
    out = torch.empty((3, K), dtype=dtype, device=cuda_device)
    z.zero1_checkpoint_unpack(k, out)
    nan = torch.isnan(out).cpu()
    want = torch.zeros((3, K), dtype=torch.bool)
    want[1, 128:256] = True
    assert torch.equal(nan, want)


# ------------------------------------------------------------- block norms ---

GATES = [None, "channel", "token", "full"]
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]
SHAPES = [(1, 1), (3, 7), (1, 256), (9, 128), (5, 500), (17, 512), (2, 513), (4, 1021), (40, 768), (3, 4096), (2, 8192),
          (2, 9000), (2, 16384)]


class Problem:
    def __init__(self, T, D, act, res, post, pre, gate, gate_act, alpha=0.5, param=BF16, seed=0):
        self.T, self.D, self.act, self.res, self.alpha, self.eps = T, D, act, res, alpha, 1e-6
        self.gate_act = gate_act
        self.y, self.x = rand((T, D), 0.7, seed + 1, act), rand((T, D), 2.0, seed + 2, res)
        self.w_post = 1 + rand((D,), 0.1, seed + 3) if post else None
        self.w_pre = 1 + rand((D,), 0.2, seed + 4) if pre else None
        self.w_post = None if self.w_post is None else self.w_post.to(param)
        self.w_pre = None if self.w_pre is None else self.w_pre.to(param)
        shape = {None: None, "channel": (D,), "token": (T, 1), "full": (T, D)}[gate]
        self.gate = None if shape is None else (0.5 + rand(shape, 0.7, seed + 5)).clamp(-3, 3).to(param)
        self.dh = rand((T, D), 1e-2, seed + 6, act) if pre else None
        self.dr = rand((T, D), 1e-2, seed + 7, res)
        self.cfg = z.BlockNorm(eps=self.eps, residual_scale=alpha, gate_act=gate_act)

    def d(self, name):
        t = getattr(self, name)
        return None if t is None else t.double()

    def forward64(self):
        return ref.forward(self.d("y"), self.d("x"), self.d("w_post"), self.d("w_pre"), self.d("gate"), self.gate_act,
                           self.alpha, self.eps)


def run_forward(p, cuda, pad=0, off=0, ckpt=True, woff=0, inplace=False):
    T, D = p.T, p.D
    o = {"r": empty(T, D, p.res, cuda, pad, off), "h": None, "rstd_post": None, "rstd_pre": None, "y8": None, "r8": None}
    x = dev(p.x, cuda, pad, off)
    if inplace:
        o["r"] = x
    if p.w_pre is not None:
        o["h"] = empty(T, D, p.act, cuda, pad, off)
        o["rstd_pre"] = torch.empty(T, device=cuda)
    if p.w_post is not None:
        o["rstd_post"] = torch.empty(T, device=cuda)
    if ckpt:
        o["y8"] = z.new_checkpoint(T, D, cuda)
        o["r8"] = z.new_checkpoint(T, D, cuda) if p.w_pre is not None else None
    z.zero1_block_norm_forward(p.cfg, dev(p.y, cuda, pad, off), x, o["r"], o["h"], o["rstd_post"], o["rstd_pre"],
                               w_post=dev(p.w_post, cuda, off=woff), w_pre=dev(p.w_pre, cuda, off=woff),
                               gate=dev(p.gate, cuda, pad if p.gate is not None and p.gate.dim() == 2 else 0, woff),
                               y8=o["y8"], r8=o["r8"])
    return o


def check_codes(k, want, rel, what):
    """A checkpoint of computed values: each value within half a code step of
    the exact one, plus the computed value's own relative error."""
    v = checkpoint_values(k)
    codes, exps = ref.pack(want)
    # 2^-4 relative is half a step of a normal code, 2^-10 scales half the
    # smallest step; a block's scale may differ by one binade at a boundary
    step = 2.0 ** (exps.double() - 127 + 1)
    step = step.repeat_interleave(128, dim=1)[:, :want.shape[1]]
    check(v, want, want.abs() * (2.0 ** -4 + rel) + step * 2.0 ** -10, what)


def check_forward(p, o):
    f = p.forward64()
    D = p.D
    rel = (D + 8) * ref.U                                   # of a statistic, and of what it scales
    if p.w_post is not None:
        check(o["rstd_post"], f["rstd_post"], f["rstd_post"] * rel, "rstd_post")
    g = ref.gate_factor(p.d("gate"), p.gate_act)
    u = f["yh"] * (p.d("w_post") if p.w_post is not None else 1.0)
    gu = (p.alpha * g * u).abs()
    r_err = gu * (rel + 4 * ref.U + (ref.SIGMOID if p.gate_act == "sigmoid" else 0)) + f["r"].abs() * ref.U
    check(o["r"], f["r"], r_err + (f["r"].abs() + r_err) * ref.half_ulp(p.res), "r")
    if o["y8"] is not None:
        check_codes(o["y8"], f["yh"], rel, "y8")
    if p.w_pre is not None:
        ms = f["r"].square().mean(1) + p.eps
        rs_rel = rel + ((f["r"].abs() * r_err).mean(1) / ms)
        check(o["rstd_pre"], f["rstd_pre"], f["rstd_pre"] * rs_rel, "rstd_pre")
        h_err = f["h"].abs() * (rs_rel[:, None] + 3 * ref.U) + r_err * f["rstd_pre"][:, None] * p.d("w_pre").abs()
        check(o["h"], f["h"], h_err + (f["h"].abs() + h_err) * ref.half_ulp(p.act), "h")
        if o["r8"] is not None:
            check_codes(o["r8"], f["rh"], float(rs_rel.max()) + 1e-5, "r8")


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("gate", GATES)
def test_forward(cuda_device, T, D, act, res, gate):
    p = Problem(T, D, act, res, True, True, gate, "sigmoid" if T % 2 else "linear")
    check_forward(p, run_forward(p, cuda_device))


@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("D", [96, 1000, 1536])
def test_forward_with_a_norm_left_out(cuda_device, post, pre, gate, D):
    p = Problem(6, D, BF16, BF16, post, pre, gate, "linear", seed=3)
    check_forward(p, run_forward(p, cuda_device))


@pytest.mark.parametrize("pad,off,woff", [(8, 0, 0), (8, 8, 0), (3, 0, 0), (0, 1, 0), (5, 3, 1), (0, 0, 1), (16, 0, 3)])
@pytest.mark.parametrize("gate", ["channel", "full"])
@pytest.mark.parametrize("param", [BF16, F32])
def test_forward_strides_and_offsets(cuda_device, pad, off, woff, gate, param):
    p = Problem(11, 1024, BF16, F32, True, True, gate, "sigmoid", param=param, seed=9)
    check_forward(p, run_forward(p, cuda_device, pad, off, woff=woff))


def test_forward_in_place_equals_out_of_place(cuda_device):
    p = Problem(37, 768, BF16, BF16, True, True, "channel", "linear")
    a, b = run_forward(p, cuda_device), run_forward(p, cuda_device, inplace=True)
    for k in ("r", "h", "rstd_pre", "rstd_post"):
        assert torch.equal(a[k], b[k])


def test_forward_zero_rows_and_empty_values(cuda_device):
    p = Problem(4, 640, BF16, BF16, True, True, "token", "linear")
    p.y[1] = 0
    p.x[1] = 0                                               # a row of zeros: 1/sqrt(eps), no NaN
    check_forward(p, run_forward(p, cuda_device))
    q = Problem(1, 640, BF16, BF16, True, True, "channel", "linear")
    e = torch.empty((0, 640), dtype=BF16, device=cuda_device)
    s = torch.empty(0, device=cuda_device)
    z.zero1_block_norm_forward(q.cfg, e, e, e, e, s, s, w_post=q.w_post.to(cuda_device), w_pre=q.w_pre.to(cuda_device),
                               gate=q.gate.to(cuda_device))


def test_forward_non_finite_rows_stay_in_their_rows(cuda_device):
    p = Problem(5, 1024, BF16, BF16, True, True, "channel", "linear")
    p.y[1, 5] = float("nan")
    p.x[3, 700] = float("inf")
    o = run_forward(p, cuda_device)
    assert not torch.isfinite(o["h"][1].float()).any() or torch.isnan(o["h"][1]).all()
    assert torch.isnan(o["h"][3, 700]) and torch.isfinite(o["h"][[0, 2, 4]].float()).all()
    assert (o["y8"].exps[:, 1] == 255).all() and (o["y8"].exps[:, 3] != 255).all()
    assert (o["r8"].exps[:, 3] == 255).any()


def run_backward(p, cuda, ckpt, pad=0, off=0, grad=F32, goff=0, accumulate=None, use_dr=True, inplace=False):
    """Kernel outputs and the 64-bit ones from the same saved activations."""
    T, D = p.T, p.D
    f = p.forward64()
    rstd = {k: None if f[k] is None else f[k].float() for k in ("rstd_post", "rstd_pre")}
    one = torch.ones(T)
    if ckpt:
        y = z.new_checkpoint(T, D, cuda)
        fill_checkpoint(y, f["yh"])
        yh = checkpoint_values(y)
        r = rh = None
        if p.w_pre is not None:
            r = z.new_checkpoint(T, D, cuda)
            fill_checkpoint(r, f["rh"])
            rh = checkpoint_values(r)
    else:
        y = dev(p.y, cuda, pad, off)
        yh = p.d("y") * (rstd["rstd_post"] if p.w_post is not None else one).double()[:, None]
        r = rh = None
        if p.w_pre is not None:
            rr = f["r"].to(p.res)
            r = dev(rr, cuda, pad, off)
            rh = rr.double() * rstd["rstd_pre"].double()[:, None]
    dr = p.dr if use_dr else None
    b = lambda t: None if t is None else t.double()  # noqa: E731
    want = ref.backward(p.d("dh"), b(dr), yh, rh, b(rstd["rstd_post"]), b(rstd["rstd_pre"]), p.d("w_post"), p.d("w_pre"),
                        p.d("gate"), p.gate_act, p.alpha)
    o = {"dy": empty(T, D, p.act, cuda, pad, off), "dx": empty(T, D, p.res, cuda, pad, off)}
    ddh, ddr = dev(p.dh, cuda, pad, off), dev(dr, cuda, pad, off)
    if inplace:
        o["dy"], o["dx"] = ddh, ddr
    start = 0.0 if accumulate is None else accumulate
    o["dw_post"] = None if p.w_post is None else dev(torch.full((D,), start, dtype=grad), cuda, off=goff)
    o["dw_pre"] = None if p.w_pre is None else dev(torch.full((D,), start, dtype=grad), cuda, off=goff)
    o["dgate"] = None
    if p.gate is not None:
        full = p.gate.shape == (T, D)
        t = torch.full(p.gate.shape, start, dtype=p.gate.dtype if full else grad)
        o["dgate"] = dev(t, cuda, pad if t.dim() == 2 else 0, goff)
    z.zero1_block_norm_backward(p.cfg, ddh, ddr, y, r, None if rstd["rstd_post"] is None else rstd["rstd_post"].to(cuda),
                                None if rstd["rstd_pre"] is None else rstd["rstd_pre"].to(cuda), o["dy"], o["dx"],
                                w_post=dev(p.w_post, cuda), w_pre=dev(p.w_pre, cuda),
                                gate=dev(p.gate, cuda, pad if p.gate is not None and p.gate.dim() == 2 else 0),
                                dw_post=o["dw_post"], dw_pre=o["dw_pre"], dgate=o["dgate"],
                                accumulate=accumulate is not None)
    return o, want


def check_backward(p, o, want, start=0.0):
    sig = ref.SIGMOID if p.gate_act == "sigmoid" else 0.0
    n = {"dx": 8, "dy": p.D + 16, "dw_pre": p.T + 4, "dw_post": p.T + 16, "dgate": 16}
    if p.gate is not None:
        n["dgate"] += p.T if p.gate.dim() == 1 else p.D if p.gate.shape[1] == 1 else 0
    for k in ("dx", "dy", "dw_pre", "dw_post", "dgate"):
        if want[k] is None:
            assert o[k] is None
            continue
        w = want[k]
        if start and (k.startswith("dw") or (k == "dgate" and p.gate.dim() == 1)):
            w = w + start
        err = want[k + "_mag"] * (n[k] * ref.U + sig * 4) + w.abs() * 2 * ref.U
        check(o[k], w, err + (w.abs() + err) * ref.half_ulp(o[k].dtype), k)


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("ckpt", [False, True])
def test_backward(cuda_device, T, D, act, res, gate, ckpt):
    p = Problem(T, D, act, res, True, True, gate, "sigmoid" if D % 2 else "linear", seed=1)
    check_backward(p, *run_backward(p, cuda_device, ckpt))


@pytest.mark.parametrize("T,D", [(700, 640), (1300, 200), (1000, 1021), (320, 9000)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_backward_more_rows_than_blocks(cuda_device, T, D, gate):
    p = Problem(T, D, BF16, BF16, True, True, gate, "sigmoid", seed=2)
    check_backward(p, *run_backward(p, cuda_device, True))


@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("ckpt", [False, True])
def test_backward_with_a_norm_left_out(cuda_device, post, pre, gate, ckpt):
    for D in (96, 1000, 1536):
        p = Problem(6, D, BF16, BF16, post, pre, gate, "linear", seed=4)
        check_backward(p, *run_backward(p, cuda_device, ckpt))


@pytest.mark.parametrize("pad,off,goff", [(8, 0, 0), (3, 1, 1), (0, 1, 0), (0, 0, 3), (8, 8, 8)])
@pytest.mark.parametrize("gate", ["channel", "token", "full"])
@pytest.mark.parametrize("grad", [BF16, F32])
def test_backward_strides_offsets_and_gradient_types(cuda_device, pad, off, goff, gate, grad):
    p = Problem(19, 1024, BF16, F32, True, True, gate, "sigmoid", seed=5)
    check_backward(p, *run_backward(p, cuda_device, False, pad, off, grad, goff))


@pytest.mark.parametrize("grad", [BF16, F32])
def test_backward_accumulates(cuda_device, grad):
    p = Problem(50, 768, BF16, BF16, True, True, "channel", "linear", seed=6)
    o, want = run_backward(p, cuda_device, True, grad=grad, accumulate=0.25)
    check_backward(p, o, want, start=0.25)


def test_backward_without_dr_and_in_place(cuda_device):
    p = Problem(50, 768, BF16, BF16, True, True, "channel", "linear", seed=7)
    check_backward(p, *run_backward(p, cuda_device, True, use_dr=False))
    a, _ = run_backward(p, cuda_device, True)
    b, _ = run_backward(p, cuda_device, True, inplace=True)
    for k in ("dx", "dy", "dw_post", "dw_pre", "dgate"):
        assert torch.equal(a[k], b[k])


def test_backward_is_reproducible(cuda_device):
    p = Problem(900, 1024, BF16, BF16, True, True, "channel", "sigmoid", seed=8)
    a, _ = run_backward(p, cuda_device, True)
    b, _ = run_backward(p, cuda_device, True)
    for k in a:
        assert torch.equal(a[k], b[k])


def test_backward_without_rows_writes_zero_sums(cuda_device):
    D = 640
    w = torch.ones(D, dtype=BF16, device=cuda_device)
    e = torch.empty((0, D), dtype=BF16, device=cuda_device)
    s = torch.empty(0, device=cuda_device)
    dw = [torch.full((D,), 3.0, dtype=BF16, device=cuda_device) for _ in range(3)]
    for acc, want in ((True, 3.0), (False, 0.0)):
        z.zero1_block_norm_backward(z.BlockNorm(), e, e, e, e, s, s, e, e, w_post=w, w_pre=w, gate=w, dw_post=dw[0],
                                    dw_pre=dw[1], dgate=dw[2], accumulate=acc)
        assert all((t == want).all() for t in dw)


# --------------------------------------------------------- weight gradient ---

def weight_grad_problem(T, N, K, seed=0):
    x = rand((T, K), 1.0, seed + 1) * torch.exp(rand((K,), 1.0, seed + 2))
    return x, rand((T, N), 1e-2, seed + 3, BF16), (1 + rand((K,), 0.2, seed + 4)).to(BF16)


def check_weight_grad(dw, dy, xv, col, T, start=0.0):
    want = dy.double().t() @ xv
    mag = dy.double().abs().t() @ xv.abs()
    if col is not None:
        want, mag = want * col.double(), mag * col.double().abs()
    want = want + start
    # the tensor cores may truncate where fp32 rounds: 2 u per addition
    err = mag * 2 * (T + 4) * ref.U + want.abs() * 2 * ref.U
    check(dw, want, err + (want.abs() + err) * ref.half_ulp(dw.dtype), "dw")


WGRAD_SHAPES = [(1, 1, 1), (1, 256, 128), (3, 5, 7), (16, 64, 128), (64, 256, 128), (65, 257, 129), (127, 384, 256),
                (128, 300, 1000), (200, 771, 640), (640, 128, 2048), (1025, 520, 136), (4100, 64, 64), (70, 1031, 515)]


@pytest.mark.parametrize("T,N,K", WGRAD_SHAPES)
@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("scaled", [False, True])
def test_weight_grad(cuda_device, T, N, K, out, scaled):
    x, dy, col = weight_grad_problem(T, N, K)
    k = z.new_checkpoint(T, K, cuda_device)
    k.exps.fill_(255)                                         # bytes past the rows hold anything
    fill_checkpoint(k, x.double())
    dw = torch.full((N, K), float("nan"), dtype=out, device=cuda_device)
    z.zero1_weight_grad(dy.to(cuda_device), k, dw, col_scale=col.to(cuda_device) if scaled else None)
    check_weight_grad(dw, dy, checkpoint_values(k), col if scaled else None, T)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,N,K", [(4500, 300, 200), (4096, 2600, 2300), (131200, 40, 72)])
def test_weight_grad_over_many_rows(cuda_device, T, N, K, out, accumulate):
    """Sums of several runs of the accumulator, in whole tiles and in parts; an
    fp32 result is near fp32 rounding however many rows there are."""
    g = torch.Generator(device=cuda_device).manual_seed(T)
    x = torch.randn((T, K), generator=g, device=cuda_device)
    dy = (torch.randn((T, N), generator=g, device=cuda_device) * 1e-2).to(BF16)
    k = z.new_checkpoint(T, K, cuda_device)
    z.zero1_checkpoint_pack(x, k)
    xv = torch.empty((T, K), device=cuda_device)
    z.zero1_checkpoint_unpack(k, xv)
    start = 0.25 if accumulate else 0.0
    dw = torch.full((N, K), start, dtype=out, device=cuda_device)
    z.zero1_weight_grad(dy, k, dw, accumulate=accumulate)
    want = dy.double().t() @ xv.double()
    err = (dw.double() - start - want).norm() / (want.norm() + start * (N * K) ** 0.5)
    # a run of 2048 rows in the tensor cores is within 1e-6 of its norm, the
    # addition of the runs within T / 2048 half ulps; bf16 adds 2^-9
    assert err <= 1e-6 + T / 2048 * ref.U + (2.0 ** -9 if out == BF16 else 0.0)


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("out", [BF16, F32])
def test_weight_grad_into_a_flat_gradient_buffer(cuda_device, pad, off, out):
    """dw and dy as views at any element offset, added to what is there."""
    T, N, K = 150, 96, 200
    x, dy, col = weight_grad_problem(T, N, K, 5)
    k = z.new_checkpoint(T, K, cuda_device)
    fill_checkpoint(k, x.double())
    flat = torch.full((off + N * K + 64,), 0.5, dtype=out, device=cuda_device)
    dw = flat[off:off + N * K].view(N, K)
    z.zero1_weight_grad(dev(dy, cuda_device, pad, off), k, dw, col_scale=col.float().to(cuda_device), accumulate=True)
    check_weight_grad(dw, dy, checkpoint_values(k), col, T, 0.5)
    assert (flat[:off] == 0.5).all() and (flat[off + N * K:] == 0.5).all()


def test_weight_grad_strided_output_leaves_the_gaps(cuda_device):
    T, N, K = 80, 70, 130
    x, dy, _ = weight_grad_problem(T, N, K, 6)
    k = z.new_checkpoint(T, K, cuda_device)
    fill_checkpoint(k, x.double())
    big = torch.full((N, K + 10), 9.0, dtype=F32, device=cuda_device)
    z.zero1_weight_grad(dy.to(cuda_device), k, big[:, :K])
    check_weight_grad(big[:, :K], dy, checkpoint_values(k), None, T)
    assert (big[:, K:] == 9.0).all()


def test_weight_grad_extreme_scales(cuda_device):
    """Checkpoint scales at both ends of their range (2^-119 .. 2^119)."""
    T, N, K = 40, 64, 256
    x, dy, _ = weight_grad_problem(T, N, K, 7)
    x = (x / x.abs().amax()).double()
    for e in (-110, -20, 20, 118):
        k = z.new_checkpoint(T, K, cuda_device)
        fill_checkpoint(k, x * 2.0 ** e * 300)
        dw = torch.empty((N, K), device=cuda_device)
        z.zero1_weight_grad(dy.to(cuda_device), k, dw)
        check_weight_grad(dw, dy, checkpoint_values(k), None, T)


def test_weight_grad_nan_block_reaches_its_columns_only(cuda_device):
    T, N, K = 90, 64, 384
    x, dy, _ = weight_grad_problem(T, N, K, 8)
    x[17, 140] = float("inf")
    k = z.new_checkpoint(T, K, cuda_device)
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    dw = torch.empty((N, K), dtype=BF16, device=cuda_device)
    z.zero1_weight_grad(dy.to(cuda_device), k, dw)
    assert torch.isnan(dw[:, 128:256]).all()
    assert torch.isfinite(dw[:, :128].float()).all() and torch.isfinite(dw[:, 256:].float()).all()


def test_weight_grad_without_rows(cuda_device):
    k = z.new_checkpoint(0, 200, cuda_device)
    dy = torch.empty((0, 96), dtype=BF16, device=cuda_device)
    dw = torch.full((96, 200), 2.0, dtype=BF16, device=cuda_device)
    z.zero1_weight_grad(dy, k, dw, accumulate=True)
    assert (dw == 2.0).all()
    z.zero1_weight_grad(dy, k, dw)
    assert (dw == 0.0).all()


@pytest.mark.parametrize("T,N,K,out", [(777, 771, 1000, F32), (16384, 512, 512, F32), (2048, 2000, 2000, BF16)])
def test_weight_grad_repeats_bit_for_bit(cuda_device, T, N, K, out):
    """Many calls in a row, with and without split tiles: no stage of a ring is
    used before it has arrived, and no wait runs out."""
    g = torch.Generator(device=cuda_device).manual_seed(T)
    x = torch.randn((T, K), device=cuda_device, generator=g)
    dy = torch.randn((T, N), device=cuda_device, generator=g).to(BF16)
    k = z.new_checkpoint(T, K, cuda_device)
    z.zero1_checkpoint_pack(x, k)
    first, dw = (torch.empty((N, K), dtype=out, device=cuda_device) for _ in range(2))
    z.zero1_weight_grad(dy, k, first)
    for _ in range(20):
        dw.zero_()
        for _ in range(50):
            z.zero1_weight_grad(dy, k, dw)
        assert torch.equal(dw, first)
    assert z.zero1_device_status() == 0


def test_weight_grad_is_reproducible(cuda_device):
    x, dy, _ = weight_grad_problem(3000, 130, 260, 9)
    k = z.new_checkpoint(3000, 260, cuda_device)
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    outs = []
    for _ in range(2):
        dw = torch.empty((130, 260), device=cuda_device)
        z.zero1_weight_grad(dy.to(cuda_device), k, dw)
        outs.append(dw)
    assert torch.equal(*outs)


# ------------------------------------------------------------------ streams ---

def test_calls_run_on_the_given_stream(cuda_device):
    """Work queued behind a busy kernel on a side stream sees inputs that are
    only written there, and workspaces belong to that stream."""
    side = torch.cuda.Stream()
    p = Problem(600, 1024, BF16, BF16, True, True, "channel", "linear", seed=11)
    a, _ = run_backward(p, cuda_device, True)
    x, dy, _ = weight_grad_problem(500, 96, 256, 12)
    k = z.new_checkpoint(500, 256, cuda_device)
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    want = torch.empty((96, 256), device=cuda_device)
    z.zero1_weight_grad(dy.to(cuda_device), k, want)
    src, ready = dy.to(cuda_device), torch.zeros((500, 96), dtype=BF16, device=cuda_device)
    k2 = z.new_checkpoint(500, 256, cuda_device)
    xs = x.to(cuda_device)
    got = torch.empty((96, 256), device=cuda_device)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        ready.copy_(src)
    z.zero1_checkpoint_pack(xs, k2, stream=side)
    z.zero1_weight_grad(ready, k2, got, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        b, _ = run_backward(p, cuda_device, True)
    side.synchronize()
    for name in a:
        assert torch.equal(a[name], b[name])


def test_pinned_host_checkpoint(cuda_device):
    """A checkpoint kept in host memory: packed and unpacked over the link."""
    x = rand((33, 1000), 1.0, 2, BF16)
    k = z.Checkpoint8(33, 1000, torch.zeros((33, 1024), dtype=torch.uint8).pin_memory(),
                      torch.zeros((8, 128), dtype=torch.uint8).pin_memory())
    z.zero1_checkpoint_pack(x.to(cuda_device), k)
    out = torch.empty((33, 1000), device=cuda_device)
    z.zero1_checkpoint_unpack(k, out)
    torch.cuda.synchronize()
    codes, exps = ref.pack(x.double())
    assert torch.equal(k.codes, codes) and torch.equal(out.double().cpu(), ref.values(codes, exps, 1000))
    assert np.array_equal(k.exps[:, :33].numpy(), exps.t().numpy())


def test_no_wait_ran_out(cuda_device):
    """The staged kernel's bounded waits all completed in the tests above."""
    assert z.zero1_device_status() == 0
