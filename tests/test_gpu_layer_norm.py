"""Layer norm with its residual on the GPU against float64, with first-order
bounds, at widths where chunks, rings and kernels change."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
U = 2.0 ** -24
SUM = 40 * U      # a row's sum: at most 40 additions deep
EPS = 1e-5
TINY = 2.0 ** -133
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]
WIDTHS = [1, 2, 7, 8, 40, 128, 200, 255, 256, 264, 512, 768, 1000, 1021, 1024, 1536, 2048, 2056, 4095, 4096, 5000, 8192, 8200, 16383, 16384]


def normal(shape, std, seed, dtype, mean=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


def within(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off their bound, at worst "
                           f"{(off / bound).nan_to_num(float('inf')).max().item():.3g} times")


class Case:
    def __init__(self, T, D, act, res, params=BF16, residual=True, ckpt=False, affine=True, mean=0.5, pad=0, offset=0):
        self.T, self.D, self.act, self.res = T, D, act, res
        self.pad, self.offset = pad, offset
        self.x = self.lay(normal((T, D), 2.0, 1, res, mean))
        self.y = self.lay(normal((T, D), 0.7, 2, act)) if residual else None
        self.w = normal((D,), 0.2, 3, params, 1.0) if affine else None
        self.b = normal((D,), 0.2, 4, params) if affine else None
        self.scale = 0.5 if residual else 1.0
        self.cfg = z.LayerNorm(eps=EPS, residual_scale=self.scale)
        self.r = self.lay(torch.zeros(T, D, dtype=res, device="cuda")) if residual else None
        self.h = self.lay(torch.zeros(T, D, dtype=act, device="cuda"))
        self.mean, self.rstd = torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda")
        self.r8 = z.new_checkpoint(T, D, "cuda") if ckpt else None

    def lay(self, t):
        """The same values with rows further apart, at an element offset."""
        if not self.pad and not self.offset:
            return t
        flat = torch.full((self.offset + t.shape[0] * (t.shape[1] + self.pad) + 8,), 3.0, dtype=t.dtype, device="cuda")
        v = flat[self.offset:self.offset + t.shape[0] * (t.shape[1] + self.pad)].view(t.shape[0], -1)[:, :t.shape[1]]
        v.copy_(t)
        return v

    def forward(self):
        z.zero1_layer_norm_forward(self.cfg, self.x, self.h, self.mean, self.rstd, w=self.w, b=self.b, y=self.y, r=self.r, r8=self.r8)

    def check_forward(self):
        r = self.x.double()
        if self.y is not None:
            r = r + self.scale * self.y.double()
        er = U * r.abs() if self.y is not None else torch.zeros_like(r)
        m = r.mean(1, keepdim=True)
        em = SUM * r.abs().mean(1, keepdim=True) + er.mean(1, keepdim=True)
        d = r - m
        ed = er + em + U * (d.abs() + em)
        var = d.square().mean(1, keepdim=True)
        ev = (2 * d.abs() * ed + ed.square()).mean(1, keepdim=True) + SUM * (var + (2 * d.abs() * ed).mean(1, keepdim=True))
        rstd = (var + EPS).rsqrt()
        rel = 0.75 * (ev / (var + EPS)) + 6 * U  # (1 + e)^-1/2 within 0.75 e for e up to 0.4; the square root's own 2 ulps
        assert bool((ev < 0.4 * (var + EPS)).all())
        rh = d * rstd
        eh = (ed * rstd + rh.abs() * rel) * 1.01 + U * rh.abs()
        within(self.mean.unsqueeze(1), m, em + U * m.abs(), "mean")
        within(self.rstd.unsqueeze(1), rstd, rstd * rel + U * rstd, "rstd")
        if self.y is not None:
            within(self.r, r, er + 1.01 * HALF[self.res] * r.abs() + TINY, "r")
        w = self.w.double() if self.w is not None else torch.ones(self.D, device="cuda", dtype=torch.float64)
        b = self.b.double() if self.b is not None else torch.zeros(self.D, device="cuda", dtype=torch.float64)
        h = rh * w + b
        within(self.h, h, eh * w.abs() + U * (h.abs() + (rh * w).abs()) + 1.01 * HALF[self.act] * h.abs() + TINY, "h")
        if self.r8 is not None:
            self.check_checkpoint(rh, eh)
        return rh

    def check_checkpoint(self, rh, eh):
        """Half a step of e4m3: 2^-4 of the value, or of the smallest normal code's,
        2^-6 of a scale that is at most amax / 224."""
        out = torch.empty(self.T, self.D, device="cuda")
        z.zero1_checkpoint_unpack(self.r8, out)
        pad = -self.D % 128
        big = torch.nn.functional.pad(rh.abs() + eh, (0, pad)).view(self.T, -1, 128).amax(2)
        scale = (big / 224).repeat_interleave(128, 1)[:, :self.D]
        within(out, rh, eh * 1.1 + 2.0 ** -4 * torch.maximum(rh.abs() + eh, 2.0 ** -6 * scale) + TINY, "r8")


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("residual,ckpt", [(True, True), (True, False), (False, False), (False, True)])
def test_forward(D, act, res, residual, ckpt):
    c = Case(37, D, act, res, BF16 if D % 2 else F32, residual, ckpt)
    c.forward()
    c.check_forward()


def check_backward(c, has_dr=True, want_dy=True, grads=F32, accumulate=False, saved=None):
    T, D = c.T, c.D
    c.forward()
    r = c.r8 if c.r8 is not None else c.r if c.r is not None else c.x
    dh, dr = c.lay(normal((T, D), 1e-2, 11, c.act)), c.lay(normal((T, D), 1e-2, 12, c.res)) if has_dr else None
    dx, dy = c.lay(torch.zeros(T, D, dtype=c.res, device="cuda")), c.lay(torch.zeros(T, D, dtype=c.act, device="cuda")) if want_dy else None
    dw, db = normal((D,), 1.0, 13, grads), normal((D,), 1.0, 14, grads)
    w0, b0 = (dw.double(), db.double()) if accumulate else (0.0, 0.0)
    z.zero1_layer_norm_backward(c.cfg, dh, dr, r, c.mean, c.rstd, dx, dy=dy, w=c.w, dw=dw, db=db, accumulate=accumulate)
    rstd = c.rstd.double().unsqueeze(1)
    if c.r8 is not None:
        v = torch.empty(T, D, device="cuda")
        z.zero1_checkpoint_unpack(c.r8, v)
        rh, eh = v.double(), 0.0
    else:
        rh = (r.double() - c.mean.double().unsqueeze(1)) * rstd
        eh = 2.1 * U * rh.abs()
    g = dh.double()
    t = g * (c.w.double() if c.w is not None else 1.0)
    et = U * t.abs()
    m1, m2 = t.mean(1, keepdim=True), (t * rh).mean(1, keepdim=True)
    e1 = (SUM * t.abs() + et).mean(1, keepdim=True) * 1.01
    e2 = ((SUM + 2 * U) * (t * rh).abs() + t.abs() * eh).mean(1, keepdim=True) * 1.01
    inner = t - m1 - rh * m2
    d = rstd * inner + (dr.double() if has_dr else 0.0)
    ed = rstd * (et + e1 + rh.abs() * e2 + eh * m2.abs() + 4 * U * (t.abs() + m1.abs() + (rh * m2).abs())) * 1.01 + 2 * U * d.abs()
    within(dx, d, ed + 1.01 * HALF[c.res] * d.abs() + TINY, "dx")
    if want_dy:
        y = c.scale * d
        within(dy, y, c.scale * ed + U * y.abs() + 1.01 * HALF[c.act] * y.abs() + TINY, "dy")
    deep = (T + 60) * U
    dww, dbb = (g * rh).sum(0) + w0, g.sum(0) + b0
    ew = deep * (g * rh).abs().sum(0) + (g.abs() * eh).sum(0)
    eb = deep * g.abs().sum(0)
    within(dw, dww, ew + 1.01 * HALF[grads] * (dww.abs() + ew) + U * dww.abs() + TINY, "dw")
    within(db, dbb, eb + 1.01 * HALF[grads] * (dbb.abs() + eb) + U * dbb.abs() + TINY, "db")


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("residual,ckpt,dr", [(True, True, True), (True, False, True), (False, False, False), (False, True, False),
                                              (True, True, False)])
def test_backward(D, act, res, residual, ckpt, dr):
    check_backward(Case(29, D, act, res, F32 if D % 2 else BF16, residual, ckpt), dr, residual, BF16 if D % 3 else F32, D % 2 == 1)


@pytest.mark.parametrize("T,D", [(1, 768), (5000, 64), (5000, 100), (2003, 1021), (3000, 4096), (700, 8192), (400, 9000)])
@pytest.mark.parametrize("act,res", TYPES)
def test_more_rows_than_blocks(T, D, act, res):
    c = Case(T, D, act, res, ckpt=D % 2 == 0)
    c.forward()
    c.check_forward()
    check_backward(c)


@pytest.mark.parametrize("pad,offset", [(8, 8), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("D", [64, 257, 1000, 8200])
@pytest.mark.parametrize("act,res", TYPES)
def test_layouts(pad, offset, D, act, res):
    for ckpt in (False, True):
        c = Case(13, D, act, res, ckpt=ckpt, pad=pad, offset=offset)
        c.forward()
        c.check_forward()
        check_backward(c)
        for t in (c.r, c.h):
            left = t.as_strided((t.shape[0], D + pad), t.stride(), t.storage_offset())[:, D:]
            assert bool((left == 3.0).all())


@pytest.mark.parametrize("act,res", TYPES)
def test_without_weights(act, res):
    c = Case(20, 300, act, res, affine=False)
    c.forward()
    c.check_forward()
    check_backward(c)


def test_a_large_mean_costs_no_bits():
    """Rows at 1000 with a spread of 1: the squares are summed about the mean."""
    c = Case(50, 1024, F32, F32, residual=False, mean=1000.0)
    c.forward()
    c.check_forward()


def test_constant_rows_and_values_that_are_not_finite():
    x = torch.ones(5, 96, device="cuda")
    x[1, 3], x[3, 95] = float("inf"), float("nan")
    h, mean, rstd = torch.empty(5, 96, device="cuda"), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    k = z.new_checkpoint(5, 96, "cuda")
    z.zero1_layer_norm_forward(z.LayerNorm(eps=EPS), x, h, mean, rstd, r8=k)
    for row in (0, 2, 4):
        assert bool((h[row] == 0).all())
    assert bool(torch.isnan(h[1]).all()) and bool(torch.isnan(h[3]).all())
    back = torch.empty(5, 96, device="cuda")
    z.zero1_checkpoint_unpack(k, back)
    assert bool(torch.isnan(back[1]).all()) and bool(torch.isnan(back[3]).all()) and bool((back[0] == 0).all())


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("D", [264, 9000])
def test_in_place(act, res, D):
    a, b = Case(33, D, act, res), Case(33, D, act, res)
    a.forward()
    b.r = b.x
    b.forward()
    assert torch.equal(a.r, b.r) and torch.equal(a.h, b.h)
    dh, dr = normal((33, D), 1e-2, 11, act), normal((33, D), 1e-2, 12, res)
    dx, dy = torch.empty_like(a.x), torch.empty_like(a.h)
    z.zero1_layer_norm_backward(a.cfg, dh, dr, a.r, a.mean, a.rstd, dx, dy=dy, w=a.w)
    z.zero1_layer_norm_backward(a.cfg, dh, dr, a.r, a.mean, a.rstd, dr, dy=dh, w=a.w)
    assert torch.equal(dx, dr) and torch.equal(dy, dh)


def test_against_differences():
    """dx, dw and db against central differences of a scalar loss in float64."""
    T, D = 3, 24
    c = Case(T, D, F32, F32, F32)
    c.forward()
    dh, dr = normal((T, D), 1.0, 11, F32), normal((T, D), 1.0, 12, F32)
    dx, dy, dw, db = torch.empty_like(c.x), torch.empty_like(c.h), torch.empty_like(c.w), torch.empty_like(c.b)
    z.zero1_layer_norm_backward(c.cfg, dh, dr, c.r, c.mean, c.rstd, dx, dy=dy, w=c.w, dw=dw, db=db)

    def loss(x, y, w, b):
        r = x + c.scale * y
        d = r - r.mean(1, keepdim=True)
        h = d * (d.square().mean(1, keepdim=True) + EPS).rsqrt() * w + b
        return (h * dh.double()).sum() + (r * dr.double()).sum()

    args = [t.double() for t in (c.x, c.y, c.w, c.b)]
    step = 1e-5
    for k, got in enumerate((dx, dy, dw, db)):
        for j in range(0, args[k].numel(), 5):
            up, down = [t.clone() for t in args], [t.clone() for t in args]
            up[k].view(-1)[j] += step
            down[k].view(-1)[j] -= step
            want = (loss(*up) - loss(*down)) / (2 * step)
            # the difference's own error: third derivatives of order 10 times step^2, and 1e-16 * loss / step
            assert abs(got.view(-1)[j].item() - want.item()) < 2e-5 * (1 + abs(want.item()))


def test_no_rows():
    D = 100
    e = torch.empty(0, D, device="cuda")
    s = torch.empty(0, device="cuda")
    z.zero1_layer_norm_forward(z.LayerNorm(), e, e.clone(), s, s.clone())
    dw, db = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    z.zero1_layer_norm_backward(z.LayerNorm(), e, None, e, s, s, e.clone(), dw=dw, db=db, accumulate=True)
    assert bool((dw == 1).all()) and bool((db == 1).all())
    z.zero1_layer_norm_backward(z.LayerNorm(), e, None, e, s, s, e.clone(), dw=dw, db=db)
    assert bool((dw == 0).all()) and bool((db == 0).all())
