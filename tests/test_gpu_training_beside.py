"""What lies beside the inputs of the training operators is NaN and reaches no
result: rows end inside wider ones, matrices inside larger buffers, at places on and
off 16-byte boundaries.  The results are those of the same values elsewhere, bit for
bit; weight and input gradients of whole numbers are the exact ones."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(autouse=True)
def no_wait_runs_out():
    yield
    assert z.zero1_device_status() == 0


def normal(*shape, std=1.0, seed=0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def blank(*shape, dtype=BF16):
    return torch.full(shape, 7.0, dtype=dtype, device="cuda")


def among(t, pad, off, fill=float("nan")):
    """The same matrix (or vector), its rows `pad` elements apart, `off` elements into a buffer of `fill`."""
    rows, cols = t.shape if t.dim() == 2 else (1, t.numel())
    flat = torch.full((off + rows * (cols + pad) + 40,), fill, dtype=t.dtype, device="cuda")
    v = flat[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(t.view(rows, cols))
    return v if t.dim() == 2 else v[0]


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    assert torch.equal(bits(a), bits(b))
    assert bool(torch.isfinite(a.float()).all())


# by rows that boxes can address, and by rows that are copied first
PLACES = [(8, 8), (16, 0), (1, 0), (3, 5), (0, 1)]


@pytest.mark.parametrize("pad,off", PLACES)
@pytest.mark.parametrize("T,D,F", [(1, 1, 1), (5, 72, 40), (40, 101, 203), (130, 200, 328), (257, 65, 130), (9, 2000, 72), (300, 64, 64)])
def test_feed_forward(T, D, F, pad, off):
    m = dict(h=normal(T, D), wg=normal(F, D, std=D ** -0.5, seed=1), wu=normal(F, D, std=D ** -0.5, seed=2),
             da=normal(T, F, std=1e-2, seed=3), dg=normal(T, F, std=1e-2, seed=4), du=normal(T, F, std=1e-2, seed=5))
    got = []
    for i in (m, {k: among(t, pad, off) for k, t in m.items()}):
        a, b, dg, du, dh, w, v = (blank(*s) for s in ((T, F), (T, F), (T, F), (T, F), (T, D), (F, D), (F, D)))
        f = blank(F, D, dtype=F32)
        z.zero1_gated_ffn_forward(i["h"], i["wg"], i["wu"], a, act="gelu")
        z.zero1_gated_ffn_backward(i["da"], i["h"], i["wg"], i["wu"], dg, du, a=b)
        z.zero1_gated_ffn_input_grad(i["dg"], i["du"], i["wg"], i["wu"], dh)
        z.zero1_weight_grad_bf16(i["dg"], i["h"], w)
        z.zero1_weight_grad_bf16(i["du"], i["h"], f)
        z.zero1_weight_grad_bf16(i["du"], i["h"], v, accumulate=True)
        got.append((a, b, dg, du, dh, w, f, v))
    for p, q in zip(*got):
        same(p, q)


@pytest.mark.parametrize("pad,off", PLACES)
@pytest.mark.parametrize("D", [1, 40, 101, 200, 1000, 1021, 2045, 4096, 5000, 9001])
@pytest.mark.parametrize("act,res", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("ckpt", [False, True])
def test_layer_norm(D, act, res, ckpt, pad, off):
    T = 23
    m = dict(x=normal(T, D, dtype=res), y=normal(T, D, seed=1, dtype=act), dh=normal(T, D, std=1e-2, seed=2, dtype=act),
             dr=normal(T, D, std=1e-2, seed=3, dtype=res), w=normal(D, seed=4), b=normal(D, seed=5))
    cfg, got = z.LayerNorm(residual_scale=0.5), []
    for fill in (0.0, float("nan")):  # (at one place, as some rows off 16-byte boundaries are summed in another order)
        i = {k: among(t, pad, off, fill) for k, t in m.items()}
        r, h, dx, dy = blank(T, D, dtype=res), blank(T, D, dtype=act), blank(T, D, dtype=res), blank(T, D, dtype=act)
        mean, rstd, dw, db = (blank(n, dtype=F32) for n in (T, T, D, D))
        k = z.new_checkpoint(T, D, "cuda") if ckpt else None
        z.zero1_layer_norm_forward(cfg, i["x"], h, mean, rstd, w=i["w"], b=i["b"], y=i["y"], r=r, r8=k)
        saved = k if ckpt else among(r, pad, off, fill)
        z.zero1_layer_norm_backward(cfg, i["dh"], i["dr"], saved, mean, rstd, dx, dy=dy, w=i["w"], dw=dw, db=db)
        got.append((r, h, mean, rstd, dx, dy, dw, db))
    for p, q in zip(*got):
        same(p, q)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_lists(dtype, off):
    sizes = [1, 7, 9, 2048, 2049, 100003, 16, 5]
    got = []
    for fill in (0.0, float("nan")):
        t = [among(normal(n, seed=n, dtype=dtype), 0, off, fill) for n in sizes]
        sumsq, norms = torch.empty(1, dtype=F64, device="cuda"), torch.empty(len(sizes), dtype=F32, device="cuda")
        z.zero1_grad_sumsq(t, sumsq, norms=norms)
        z.zero1_grad_clip(t, sumsq, 0.5 * sumsq.item() ** 0.5)
        got.append((sumsq, norms, *t))
    for p, q in zip(*got):
        same(p, q)


@pytest.mark.parametrize("n,M,align", [(5, 3, 8), (1000, 2, 128), (10007, 4, 8), (4099, 5, 1)])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_clipped_step(n, M, align, off):
    plan = z.zero1_plan(n, M, align)
    hp = z.AdamW(global_batch=64, step=3)
    P = plan.padded_n
    grads = [normal(n, seed=10 + k) for k in range(M)]
    state = [normal(P, std=s, seed=20 + k, dtype=F32) for k, s in enumerate((0.02, 1e-4, 1e-3))]
    state[2].square_()
    for s in state:
        s[n:] = 0
    got = []
    for lay in (lambda t: t.clone(), lambda t: among(t, 0, off)):
        g, s, p = [lay(t) for t in grads], [lay(t) for t in state], blank(n)
        q, sums = torch.empty(1, dtype=F64, device="cuda"), blank(P, dtype=F32)
        z.zero1_shard_grad_sumsq(plan, 0, M, g, hp, q, sums=sums)
        total = torch.tensor([4.0], dtype=F64, device="cuda") if not got else got[0][-1]
        z.zero1_step_clipped(plan, 0, M, g, *s, p, hp, total, 0.5, sums=sums)
        kept = [t.clone() for t in (*s, p)]
        s, p2 = [lay(t) for t in state], blank(n)
        z.zero1_step_clipped(plan, 0, M, g, *s, p2, hp, total, 0.5)
        assert abs(q.item() - sum(t.double() for t in g).square().sum().item() / 64 ** 2) <= 1e-5 * q.item()
        got.append((*kept, *s, p2, sums, total))
    for a, b in zip(*got):
        same(a, b)


def whole(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-4, 5, (rows, cols), generator=g, device="cuda").to(BF16)


# contractions in one run and in several, tiles done whole and split, edges on and off 16 bytes
WHOLE = [(100, 300, 260), (777, 771, 1000), (2048, 512, 512), (5000, 2560, 2560), (5000, 2555, 2557), (9000, 300, 200), (2200, 70, 130)]


@pytest.mark.parametrize("T,N,K", WHOLE)
@pytest.mark.parametrize("off", [0, 1, 4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weight_gradients_of_whole_numbers(T, N, K, off, dtype):
    dy, x = whole(T, N, 1), whole(T, K, 2)
    exact = dy.double().t() @ x.double()
    assert exact.abs().max() < 2 ** 24
    flat = torch.full((off + N * K + 8,), 7.0, dtype=dtype, device="cuda")
    dw = flat[off:off + N * K].view(N, K)
    z.zero1_weight_grad_bf16(dy, x, dw)
    assert torch.equal(dw, exact.to(dtype))
    start = (torch.randint(-100, 100, (N, K), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * 2 ** 8).to(dtype)
    dw.copy_(start)
    z.zero1_weight_grad_bf16(dy, x, dw, accumulate=True)
    assert torch.equal(dw, (start.double() + exact).to(dtype))
    # nothing is added to subnormal, smallest and largest values
    e = torch.randint(-148, 127, (N, K), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").double()
    start = (torch.exp2(e) * 1.5).float().to(dtype)
    dw.copy_(start)
    z.zero1_weight_grad_bf16(torch.zeros_like(dy), x, dw, accumulate=True)
    assert torch.equal(bits(dw), bits(start))
    assert bool((flat[:off] == 7).all() and (flat[off + N * K:] == 7).all())


@pytest.mark.parametrize("T,D,F", [(1, 1, 1), (3, 300, 260), (777, 771, 1000), (300, 512, 4100), (5, 8, 9000), (2300, 256, 1216)])
def test_input_gradients_of_whole_numbers(T, D, F):
    dg, du, wg, wu = whole(T, F, 1), whole(T, F, 2), whole(F, D, 3), whole(F, D, 4)
    dh = blank(T, D)
    z.zero1_gated_ffn_input_grad(dg, du, wg, wu, dh)
    assert torch.equal(dh, (dg.double() @ wg.double() + du.double() @ wu.double()).to(BF16))
