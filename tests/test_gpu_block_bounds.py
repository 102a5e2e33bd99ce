"""The block norms against the 64-bit formulas within first-order bounds
(block_bounds.py), every output of both directions, with few rows and with many
more rows than blocks.  The formulas run on the GPU in fp64."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
import block_bounds as bb
import block_reference as ref

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32)]
EPS = 1e-6


def placed(t, pad, off):
    """A copy of a matrix with rows `pad` elements apart, `off` into its buffer, NaN around it."""
    T, D = t.shape
    big = torch.full((off + T * (D + pad) + 8,), float("nan"), dtype=t.dtype, device=t.device)
    v = big[off:off + T * (D + pad)].view(T, D + pad)[:, :D]
    v.copy_(t)
    return v


def code_values(k, T, D):
    """fp64 values of a checkpoint."""
    e = k.exps[:, :T].t().double() - 127
    v = k.codes.view(torch.float8_e4m3fn).double().view(T, -1, 128) * torch.exp2(e)[:, :, None]
    return v.view(T, -1)[:, :D]


def assert_within(got, want, err, what):
    bad = bb.outside(got, want, err, got.dtype)
    assert got.shape == want.shape and not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


class Case:
    def __init__(self, cuda, T, D, act, res, gate, gate_act="linear", post=True, pre=True, ckpt=False, pad=0, off=0,
                 inplace=False, grad=F32):
        self.__dict__.update(locals())
        g = torch.Generator(device=cuda).manual_seed(T * 7 + D)
        r = lambda *s: torch.randn(s, generator=g, device=cuda)  # noqa: E731
        put = lambda t: placed(t, pad, off)  # noqa: E731
        self.put = put
        self.y, self.x = put((r(T, D) * 0.7).to(act)), put((r(T, D) * 2).to(res))
        self.w_post = (1 + 0.1 * r(D)).to(BF16) if post else None
        self.w_pre = (1 + 0.2 * r(D)).to(BF16) if pre else None
        shape = {None: None, "channel": (D,), "token": (T, 1), "full": (T, D)}[gate]
        self.gates = None if shape is None else (0.5 + 0.7 * r(*shape)).to(BF16)
        if gate == "full":
            self.gates = put(self.gates)
        # along the rows, so that the rows' means matter
        self.dh = put((1e-2 * (r(T, D) + self.x.float())).to(act)) if pre else None
        self.dr = put((1e-2 * (r(T, D) + self.y.float())).to(res))
        self.cfg = z.BlockNorm(eps=EPS, residual_scale=0.5, gate_act=gate_act)
        self.weights = dict(w_post=self.w_post, w_pre=self.w_pre, gate=self.gates)
        d = lambda t: None if t is None else t.double()  # noqa: E731
        self.w64 = (d(self.w_post), d(self.w_pre), d(self.gates))
        self.f = ref.forward(d(self.y), d(self.x), *self.w64, gate_act, 0.5, EPS)

    def empty(self, dtype):
        return self.put(torch.full((self.T, self.D), float("nan"), dtype=dtype, device=self.cuda))

    def stat(self, there):
        return torch.full((self.T,), float("nan"), device=self.cuda) if there else None

    def forward(self):
        T, D, f = self.T, self.D, self.f
        x = self.put(self.x) if self.inplace else self.x
        r = x if self.inplace else self.empty(self.res)
        h = self.empty(self.act) if self.pre else None
        rstd_post, rstd_pre = self.stat(self.post), self.stat(self.pre)
        y8 = z.new_checkpoint(T, D, self.cuda) if self.ckpt else None
        r8 = z.new_checkpoint(T, D, self.cuda) if self.ckpt and self.pre else None
        z.zero1_block_norm_forward(self.cfg, self.y, x, r, h, rstd_post, rstd_pre, y8=y8, r8=r8, **self.weights)
        err = bb.forward_bounds(f, *self.w64, self.gate_act, 0.5, EPS, D)
        assert_within(r, f["r"], err["r"], "r")
        if self.post:
            assert_within(rstd_post, f["rstd_post"], err["rstd_post"], "rstd_post")
        if self.pre:
            assert_within(rstd_pre, f["rstd_pre"], err["rstd_pre"], "rstd_pre")
            assert_within(h, f["h"], err["h"], "h")
        if y8 is not None:
            self.codes_within(y8, f["yh"], f["yh"].abs() * err["yh_rel"], "y8")
        if r8 is not None:
            self.codes_within(r8, f["rh"], f["rh"].abs() * err["rh_rel"] + err["rh_abs"], "r8")

    def codes_within(self, k, want, err, what):
        """Half a code's step off the value that was packed: 2^-4 of it, or
        2^-10 of the block's scale, which may be one binade up at a boundary."""
        v = code_values(k, self.T, self.D)
        pad = ref.up(self.D) - self.D
        amax = torch.nn.functional.pad(want + 0, (0, pad)).view(self.T, -1, 128).abs().amax(2)
        scale = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(1e-30) / 448)) + 1).repeat_interleave(128, 1)[:, :self.D]
        assert ((v - want).abs() <= (want.abs() + err) * 2.0 ** -4 + err + scale * 2.0 ** -10).all(), what
        if pad:
            assert (k.codes[:, self.D:] == 0).all(), what

    def backward(self):
        T, D, f = self.T, self.D, self.f
        rstd_post = f["rstd_post"].float() if self.post else None
        rstd_pre = f["rstd_pre"].float() if self.pre else None
        if self.ckpt:
            y, r, rh = z.new_checkpoint(T, D, self.cuda), None, None
            z.zero1_checkpoint_pack(f["yh"].float(), y)
            yh = code_values(y, T, D)
            if self.pre:
                r = z.new_checkpoint(T, D, self.cuda)
                z.zero1_checkpoint_pack(f["rh"].float(), r)
                rh = code_values(r, T, D)
        else:
            y, r, rh = self.y, None, None
            yh = self.y.double() * rstd_post.double()[:, None] if self.post else self.y.double()
            if self.pre:
                r = self.put(f["r"].to(self.res))
                rh = r.double() * rstd_pre.double()[:, None]
        dh, dr = self.dh, self.dr
        dy, dx = self.empty(self.act), self.empty(self.res)
        if self.inplace:
            dx = dr = self.put(dr)
            if self.pre:
                dy = dh = self.put(dh)
        sums = lambda there: torch.full((D,), float("nan"), dtype=self.grad, device=self.cuda) if there else None  # noqa: E731
        dw_post, dw_pre = sums(self.post), sums(self.pre)
        dgate = None
        if self.gates is not None:
            full = self.gates.shape == (T, D)     # (a token's gate too, where a row has one column)
            dgate = torch.full(self.gates.shape, float("nan"), device=self.cuda, dtype=BF16 if full else self.grad)
        z.zero1_block_norm_backward(self.cfg, dh, dr, y, r, rstd_post, rstd_pre, dy, dx, dw_post=dw_post, dw_pre=dw_pre,
                                    dgate=dgate, **self.weights)
        d = lambda t: None if t is None else t.double()  # noqa: E731
        args = (d(self.dh), d(self.dr), yh, rh, d(rstd_post), d(rstd_pre), *self.w64, self.gate_act, 0.5)
        want = ref.backward(*args)
        err = bb.backward_bounds(want, *args)
        for k, got in (("dx", dx), ("dy", dy), ("dw_post", dw_post), ("dw_pre", dw_pre), ("dgate", dgate)):
            if got is not None:
                assert_within(got, want[k], err[k], k)

    def both(self):
        self.forward()
        self.backward()


SHAPES = [(1, 1), (3, 7), (1, 256), (9, 128), (5, 500), (17, 512), (2, 513), (4, 1021), (40, 768), (6, 1280), (6, 1600),
          (3, 2048), (3, 4096), (3, 5120), (2, 8192), (2, 9000), (2, 16384)]
# far more rows than the 2432 to 152 blocks that are resident
MANY = [(26000, 250), (13000, 500), (5000, 768), (5000, 1021), (5000, 1600), (2500, 4096), (1500, 5120), (1500, 8192),
        (900, 9000), (700, 16384)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("ckpt", [False, True])
def test_few_rows(cuda_device, T, D, act, res, gate, ckpt):
    Case(cuda_device, T, D, act, res, gate, "sigmoid" if D % 2 else "linear", ckpt=ckpt).both()


@pytest.mark.parametrize("T,D", MANY)
@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("ckpt", [False, True])
def test_many_rows(cuda_device, T, D, act, res, gate, ckpt):
    Case(cuda_device, T, D, act, res, gate, "sigmoid" if T % 1000 else "linear", ckpt=ckpt).both()


@pytest.mark.parametrize("T,D", [(5000, 768), (5000, 1021), (1500, 8192), (900, 9000)])
@pytest.mark.parametrize("post,pre", [(True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("ckpt", [False, True])
def test_many_rows_with_a_norm_left_out(cuda_device, T, D, post, pre, gate, ckpt):
    Case(cuda_device, T, D, BF16, F32, gate, "sigmoid", post, pre, ckpt).both()


@pytest.mark.parametrize("T,D", [(5000, 768), (5000, 1021), (2500, 4096), (900, 9000)])
@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("pad,off", [(8, 8), (3, 1), (0, 1)])
@pytest.mark.parametrize("gate", ["channel", "full"])
@pytest.mark.parametrize("inplace", [False, True])
def test_many_rows_strided_and_in_place(cuda_device, T, D, act, res, pad, off, gate, inplace):
    Case(cuda_device, T, D, act, res, gate, "linear", pad=pad, off=off, inplace=inplace, grad=BF16).both()


def test_forward_repeats_bit_for_bit(cuda_device):
    """Many calls in a row with more rows than blocks give the same bits."""
    c = Case(cuda_device, 8192, 4096, BF16, BF16, "channel", ckpt=True)
    outs = []
    for _ in range(20):
        r, h, a, b = c.empty(BF16), c.empty(BF16), c.stat(True), c.stat(True)
        y8, r8 = (z.new_checkpoint(c.T, c.D, cuda_device) for _ in range(2))
        z.zero1_block_norm_forward(c.cfg, c.y, c.x, r, h, a, b, y8=y8, r8=r8, **c.weights)
        outs.append((r, h, a, b, y8.codes, r8.codes, y8.exps[:, :c.T], r8.exps[:, :c.T]))
        assert all(torch.equal(p, q) for p, q in zip(outs[0], outs[-1]))
        outs = outs[:1]
