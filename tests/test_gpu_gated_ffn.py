"""The gated feed-forward block and the bf16 weight gradient on the GPU against
float64, at the sizes, strides and values where tiles, splits and copies go wrong."""
import pytest
import torch

import ffn_reference as ref
import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CANARY = 7.0

# rows, width, inner width: single elements, less than a tile, tile edges and one
# beyond, several tiles, contractions that are split over blocks, odd widths
SIZES = [(1, 1, 1), (1, 64, 64), (2, 8, 8), (5, 72, 40), (129, 200, 264), (256, 128, 256), (257, 65, 130), (128, 64, 128),
         (300, 1000, 771), (512, 768, 2048), (3, 4096, 512), (64, 8192, 200), (1000, 512, 1537), (1, 2048, 4100),
         (2300, 256, 1216), (640, 1408, 5000)]


@pytest.fixture(autouse=True)
def no_wait_runs_out():
    yield
    assert z.zero1_device_status() == 0


def normal(rows, cols, std, seed, dtype=BF16, ld=None, offset=0):
    """A [rows, cols] view of normal draws with rows `ld` apart, `offset` elements
    into a buffer whose other elements are CANARY."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ld = cols if ld is None else ld
    flat = torch.full((offset + rows * ld + 64,), CANARY, device="cuda", dtype=dtype)
    v = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    v.copy_(torch.randn(rows, cols, generator=g, device="cuda") * std)
    v.flat = flat
    return v


def blank(rows, cols, dtype=BF16, ld=None, offset=0):
    ld = cols if ld is None else ld
    flat = torch.full((offset + rows * ld + 64,), CANARY, device="cuda", dtype=dtype)
    v = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    v.flat = flat
    return v


def untouched(v):
    """What lies around a view's rows is what it was."""
    flat = v.flat.clone()
    flat.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(CANARY)
    assert bool((flat == CANARY).all())


def block(T, D, F, seed=0, **kw):
    return (normal(T, D, 1.0, seed, **kw), normal(F, D, D ** -0.5, seed + 1, **kw), normal(F, D, D ** -0.5, seed + 2, **kw))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_forward(T, D, F, act):
    h, wg, wu = block(T, D, F)
    a = blank(T, F)
    z.zero1_gated_ffn_forward(h, wg, wu, a, act=act)
    ref.check(a, ref.forward(h, wg, wu, act), "a")
    untouched(a)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,D,F", SIZES)
def test_backward(T, D, F, act):
    h, wg, wu = block(T, D, F)
    da = normal(T, F, 1e-3, 5)
    a, dg, du = blank(T, F), blank(T, F), blank(T, F)
    z.zero1_gated_ffn_backward(da, h, wg, wu, dg, du, a=a, act=act)
    g, u = ref.backward(da, h, wg, wu, act)
    ref.check(dg, g, "dg")
    ref.check(du, u, "du")
    ref.check(a, ref.forward(h, wg, wu, act), "a")
    for v in (a, dg, du):
        untouched(v)
    again = blank(T, F)
    z.zero1_gated_ffn_backward(da, h, wg, wu, da, again, act=act)  # dg in the place of da, no a
    assert torch.equal(da, dg) and torch.equal(again, du)


@pytest.mark.parametrize("T,D,F", SIZES)
def test_input_grad(T, D, F):
    _, wg, wu = block(T, D, F)
    dg, du = normal(T, F, 1e-3, 6), normal(T, F, 1e-3, 7)
    dh = blank(T, D)
    z.zero1_gated_ffn_input_grad(dg, du, wg, wu, dh)
    ref.check(dh, ref.input_grad(dg, du, wg, wu), "dh")
    untouched(dh)


WEIGHTS = [(0, 5, 7), (1, 1, 1), (1, 300, 520), (7, 8, 8), (64, 256, 256), (65, 257, 255), (777, 771, 1000), (2048, 128, 64),
           (2049, 130, 70), (5000, 300, 200), (20000, 64, 32), (9000, 2600, 2500), (1500, 5000, 4100)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("T,N,K", WEIGHTS)
def test_weight_grad(T, N, K, dtype, accumulate):
    dy, x = normal(T, N, 1e-3, 8), normal(T, K, 1.0, 9)
    dw = normal(N, K, 1e-2, 10, dtype=dtype)
    start = dw.clone()
    z.zero1_weight_grad_bf16(dy, x, dw, accumulate=accumulate)
    ref.check(dw, ref.weight_grad(dy, x, dtype, start if accumulate else None), "dw")
    untouched(dw)


# element offsets and row strides: on 16-byte boundaries in a wider matrix, off them, odd
LAYOUTS = [dict(ld=344, offset=8), dict(ld=341, offset=0), dict(ld=336, offset=1), dict(ld=339, offset=3), dict(ld=340, offset=4)]


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D,F", [(200, 330), (330, 200), (328, 328), (321, 323)])
def test_layouts(layout, D, F):
    T = 150
    h, wg, wu = block(T, D, F, **layout)
    da = normal(T, F, 1e-3, 5, **layout)
    a, dg, du, dh = (blank(T, n, **layout) for n in (F, F, F, D))
    z.zero1_gated_ffn_forward(h, wg, wu, a)
    want = ref.forward(h, wg, wu, "silu")
    ref.check(a, want, "a")
    a.fill_(0)
    z.zero1_gated_ffn_backward(da, h, wg, wu, dg, du, a=a)
    ref.check(a, want, "a again")
    for got, w in zip((dg, du), ref.backward(da, h, wg, wu, "silu")):
        ref.check(got, w, "dg, du")
    z.zero1_gated_ffn_input_grad(dg, du, wg, wu, dh)
    ref.check(dh, ref.input_grad(dg, du, wg, wu), "dh")
    for dtype in (BF16, F32):
        dw = blank(F, D, dtype=dtype, **layout)
        z.zero1_weight_grad_bf16(dg, h, dw)
        ref.check(dw, ref.weight_grad(dg, h, dtype), "dw")
        untouched(dw)
    for v in (a, dg, du, dh):
        untouched(v)


def test_an_odd_width_in_a_wider_matrix_reads_none_of_what_is_beside_it():
    T, D, F = 40, 101, 203
    h, wg, wu = block(T, D, F, ld=208)
    for v in (h, wg, wu):
        v.flat[v.flat == CANARY] = float("nan")
    a = blank(T, F)
    z.zero1_gated_ffn_forward(h, wg, wu, a)
    ref.check(a, ref.forward(h, wg, wu, "silu"), "a")


def test_rows_that_repeat():
    """Inputs may have a row stride of 0: the same row again."""
    F, D = 130, 72
    _, wg, wu = block(1, D, F)
    h = normal(1, D, 1.0, 3).expand(50, D)
    a = blank(50, F)
    z.zero1_gated_ffn_forward(h, wg, wu, a)
    ref.check(a, ref.forward(h, wg, wu, "silu"), "a")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_extreme_values(act):
    """Pre-activations from -1e30 to 1e30, subnormal ones and zeros; an Inf or a NaN
    reaches its own row only."""
    D = 8
    points = [0.0, -0.0, 1e-40, -1e-40, 1e-20, 0.5, -0.5, -1.278, 3.0, -3.0, -8.0, 20.0, -20.0, -60.0, -87.0, -88.5, -90.0,
              -100.0, -104.0, 88.0, 100.0, 1e4, -1e4, 1e10, -1e10, 1e30, -1e30]
    h = torch.zeros(len(points) + 3, D, device="cuda", dtype=BF16)
    h[:len(points), 0] = torch.tensor(points, device="cuda").to(BF16)
    h[-3:, 0] = torch.tensor([float("inf"), float("-inf"), float("nan")], device="cuda").to(BF16)
    h[:, 1] = 1.0
    wg, wu = torch.zeros(16, D, device="cuda", dtype=BF16), torch.zeros(16, D, device="cuda", dtype=BF16)
    wg[:, 0], wu[:, 1] = 1.0, 2.0
    T = h.shape[0]
    a, da, dg, du = blank(T, 16), torch.full((T, 16), 0.25, device="cuda", dtype=BF16), blank(T, 16), blank(T, 16)
    z.zero1_gated_ffn_backward(da, h, wg, wu, dg, du, a=a, act=act)
    n = len(points)
    ref.check(a[:n], ref.forward(h[:n], wg, wu, act), "a")
    g, u = ref.backward(da[:n], h[:n], wg, wu, act)
    ref.check(du[:n], u, "du")
    ok = (h[:n, 0].float().abs() < 1e9)  # (g^2 of gelu's slope leaves fp32 beyond)
    ref.check(dg[:n][ok], tuple(t[ok] for t in g), "dg")
    assert not torch.isfinite(a[-3:].float()).any(dim=1).any() or not torch.isfinite(a[-1].float()).any()
    assert torch.isnan(a[-1].float()).all() and torch.isnan(dg[-1].float()).all() and torch.isnan(du[-1].float()).all()


def test_no_rows():
    _, wg, wu = block(1, 64, 96)
    e = lambda n: torch.empty(0, n, device="cuda", dtype=BF16)  # noqa: E731
    z.zero1_gated_ffn_forward(e(64), wg, wu, e(96))
    z.zero1_gated_ffn_backward(e(96), e(64), wg, wu, e(96), e(96))
    z.zero1_gated_ffn_input_grad(e(96), e(96), wg, wu, e(64))
