"""Inputs that the header allows and programs hand over: rows that repeat or
overlap, one tensor in two places of a call, weights and gradients at odd places of
a flat buffer, checkpoints and rows inside larger ones.  Results are those of rows
that lie apart, bit for bit."""
import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
from test_gpu_block_strides import apart, rows

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
CUDA = "cuda"


@pytest.fixture(autouse=True)
def no_wait_runs_out():
    yield
    assert z.zero1_device_status() == 0


def normal(*shape, std=1.0, seed=0, dtype=BF16):
    g = torch.Generator(device=CUDA).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=CUDA) * std).to(dtype)


def blank(*shape, dtype=BF16):
    return torch.full(shape, 7.0, dtype=dtype, device=CUDA)


# rows, width, row stride, element offset: once repeated, once overlapping by whole 16-byte
# steps (boxes can address them), once by odd ones
OVERLAPS = [(300, 512, 0, 0), (300, 512, 8, 0), (300, 512, 64, 8), (300, 512, 3, 0), (300, 511, 7, 1), (40, 72, 16, 0), (700, 264, 8, 0)]


@pytest.mark.parametrize("T,D,ld,off", OVERLAPS)
def test_feed_forward_of_rows_that_repeat_or_overlap(T, D, ld, off):
    F = 200
    wg, wu = normal(F, D, std=0.05, seed=1), normal(F, D, std=0.05, seed=2)
    h = rows(T, D, ld, BF16, CUDA, 3, off)
    da = rows(T, F, min(ld, F), BF16, CUDA, 4, off)
    got = []
    for c in (lambda t: t, apart):
        a, again, dg, du = (blank(T, F) for _ in range(4))
        z.zero1_gated_ffn_forward(c(h), wg, wu, a)
        z.zero1_gated_ffn_backward(c(da), c(h), wg, wu, dg, du, a=again, act="gelu")
        got.append((a, again, dg, du))
    for p, q in zip(*got):
        assert torch.equal(p, q)
    # the same rows as weights, and as gradients of the projections
    x = normal(50, D, seed=5)
    got = []
    for c in (lambda t: t, apart):
        a = blank(50, T)
        z.zero1_gated_ffn_forward(x, c(h), c(h), a)
        dh, g = blank(T, 40), normal(D, 40, std=0.05, seed=6)
        z.zero1_gated_ffn_input_grad(c(h), c(h), g, g, dh)
        got.append((a, dh))
    for p, q in zip(*got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("T,D,ld,off", OVERLAPS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_weight_gradient_of_rows_that_repeat_or_overlap(T, D, ld, off, dtype):
    dy, x = rows(T, D, ld, BF16, CUDA, 7, off), normal(T, 136, seed=8)
    for a, b in ((dy, x), (x, dy), (dy, dy)):  # (the last: the same tensor twice)
        p, q = (blank(a.shape[1], b.shape[1], dtype=dtype) for _ in range(2))
        z.zero1_weight_grad_bf16(a, b, p)
        z.zero1_weight_grad_bf16(apart(a), apart(b), q)
        assert torch.equal(p, q)


@pytest.mark.parametrize("T,D,ld,off", [(300, 1024, 0, 0), (300, 1024, 8, 0), (300, 1024, 1, 0), (300, 1021, 7, 1), (40, 9000, 0, 0),
                                        (40, 9000, 4, 3), (300, 200, 64, 0)])
@pytest.mark.parametrize("act,res", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_layer_norm_of_rows_that_repeat_or_overlap(T, D, ld, off, act, res):
    y, x = rows(T, D, ld, act, CUDA, 2, off), rows(T, D, ld, res, CUDA, 3, off)
    dh, dr = rows(T, D, ld, act, CUDA, 4, off), rows(T, D, ld, res, CUDA, 5, off)
    w = normal(D, std=0.2, seed=6) + 1
    cfg, got = z.LayerNorm(residual_scale=0.5), []
    for c in (lambda t: t, apart):
        r, h, dx, dy = blank(T, D, dtype=res), blank(T, D, dtype=act), blank(T, D, dtype=res), blank(T, D, dtype=act)
        a, b, dw, db = (blank(n, dtype=F32) for n in (T, T, D, D))
        z.zero1_layer_norm_forward(cfg, c(x), h, a, b, w=w, b=w, y=c(y), r=r)
        z.zero1_layer_norm_backward(cfg, c(dh), c(dr), c(x), a, b, dx, dy=dy, w=w, dw=dw, db=db)
        got.append((r, h, a, b, dx, dy, dw, db))
    for k, (p, q) in enumerate(zip(*got)):
        assert torch.equal(p, q), k


@pytest.mark.parametrize("T,D,F", [(40, 64, 96), (300, 200, 333), (9, 4096, 136)])
def test_one_tensor_in_two_places(T, D, F):
    h, w, da = normal(T, D), normal(F, D, std=D ** -0.5, seed=1), normal(T, F, std=1e-2, seed=2)
    got = []
    for two in (w, w.clone()):
        a, dg, du, dh = blank(T, F), blank(T, F), blank(T, F), blank(T, D)
        z.zero1_gated_ffn_forward(h, w, two, a)
        z.zero1_gated_ffn_backward(da, h, w, two, dg, du)
        z.zero1_gated_ffn_input_grad(da, da if two is w else da.clone(), w, two, dh)
        got.append((a, dg, du, dh))
    for p, q in zip(*got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("D", [8, 200, 1000, 1021, 4096, 9000])
@pytest.mark.parametrize("params", [BF16, F32])
@pytest.mark.parametrize("grads", [BF16, F32])
def test_layer_norm_vectors_at_odd_places_and_each_left_out(D, params, grads):
    """w and b anywhere in a flat buffer, dw and db too; each of the four with and
    without the others gives the same; what lies beside the gradients stays."""
    T, off = 45, 3
    x, dh = normal(T, D, seed=1), normal(T, D, std=1e-2, seed=2)
    w, b = normal(D, std=0.2, seed=3, dtype=params) + 1, normal(D, std=0.2, seed=4, dtype=params)
    flat = normal(2 * D + 9, seed=5, dtype=params)
    wo, bo = flat[off:off + D], flat[off + D + 2:off + 2 * D + 2]
    wo.copy_(w), bo.copy_(b)
    mean, rstd = blank(T, dtype=F32), blank(T, dtype=F32)
    h = [blank(T, D) for _ in range(4)]
    cfg, one, none = z.LayerNorm(), torch.ones_like(w), torch.zeros_like(b)
    z.zero1_layer_norm_forward(cfg, x, h[0], mean, rstd, w=w, b=b)
    z.zero1_layer_norm_forward(cfg, x, h[1], mean, rstd, w=wo, b=bo)
    assert torch.equal(h[0], h[1])
    for kw, full in ((dict(w=wo), (w, none)), (dict(b=bo), (one, b)), ({}, (one, none))):
        z.zero1_layer_norm_forward(cfg, x, h[2], mean, rstd, **kw)
        z.zero1_layer_norm_forward(cfg, x, h[3], mean, rstd, w=full[0], b=full[1])
        assert torch.equal(h[2], h[3])
    dx, dx2, dw, db = blank(T, D), blank(T, D), blank(D, dtype=grads), blank(D, dtype=grads)
    z.zero1_layer_norm_backward(cfg, dh, None, x, mean, rstd, dx, w=w, dw=dw, db=db)
    buf = blank(2 * D + 9, dtype=grads)
    z.zero1_layer_norm_backward(cfg, dh, None, x, mean, rstd, dx2, w=wo, dw=buf[off:off + D], db=buf[off + D + 2:off + 2 * D + 2])
    assert torch.equal(dx, dx2) and torch.equal(buf[off:off + D], dw) and torch.equal(buf[off + D + 2:off + 2 * D + 2], db)
    assert bool((buf[:off] == 7).all() and (buf[off + D:off + D + 2] == 7).all() and (buf[off + 2 * D + 2:] == 7).all())
    for kw, want in ((dict(dw=buf[1:D + 1]), dw), (dict(db=buf[1:D + 1]), db)):
        buf.fill_(7.0)
        z.zero1_layer_norm_backward(cfg, dh, None, x, mean, rstd, dx2, w=w, **kw)
        assert torch.equal(buf[1:D + 1], want) and torch.equal(dx, dx2)
        assert bool((buf[:1] == 7).all() and (buf[D + 1:] == 7).all())


@pytest.mark.parametrize("T,D", [(45, 200), (5, 1000), (130, 4096), (7, 9000)])
@pytest.mark.parametrize("act,res", [(BF16, BF16), (BF16, F32), (F32, F32)])
def test_layer_norm_checkpoint_in_a_larger_store(T, D, act, res):
    wide, high = -(-D // 128) * 128, -(-T // 128) * 128
    x = normal(T, D, seed=1, dtype=res)
    codes, exps = (torch.full(s, 0x5A, dtype=torch.uint8, device=CUDA) for s in ((T + 2, wide + 256), (wide // 128 + 1, high + 128)))
    big = z.Checkpoint8(T, D, codes[1:T + 1, 128:128 + wide], exps[:wide // 128, :high])
    near = z.new_checkpoint(T, D, CUDA)
    h, h2, stats = blank(T, D, dtype=act), blank(T, D, dtype=act), [blank(T, dtype=F32) for _ in range(2)]
    z.zero1_layer_norm_forward(z.LayerNorm(), x, h, *stats, r8=near)
    z.zero1_layer_norm_forward(z.LayerNorm(), x, h2, *stats, r8=big)
    assert torch.equal(h, h2) and torch.equal(big.codes, near.codes) and torch.equal(big.exps[:, :T], near.exps[:, :T])
    left = codes.clone()
    left[1:T + 1, 128:128 + wide] = 0x5A
    assert bool((left == 0x5A).all()) and bool((exps[:, high:] == 0x5A).all()) and bool((exps[wide // 128:] == 0x5A).all())
    dh, dx = normal(T, D, std=1e-2, seed=2, dtype=act), [blank(T, D, dtype=res) for _ in range(2)]
    g = [blank(D, dtype=F32) for _ in range(4)]
    z.zero1_layer_norm_backward(z.LayerNorm(), dh, None, near, *stats, dx[0], dw=g[0], db=g[1])
    z.zero1_layer_norm_backward(z.LayerNorm(), dh, None, big, *stats, dx[1], dw=g[2], db=g[3])
    assert torch.equal(dx[0], dx[1]) and torch.equal(g[0], g[2]) and torch.equal(g[1], g[3])


def test_outputs_of_the_clipped_step_each_its_own_way():
    """master in place, m and v to other buffers, and every other mixture."""
    n, M = 70001, 4
    plan = z.zero1_plan(n, M, 8)
    P = plan.padded_n
    hp = z.AdamW(global_batch=64, step=3)
    grads = [normal(n, seed=10 + k) for k in range(M)]
    state = [normal(P, std=s, seed=20 + k, dtype=F32) for k, s in enumerate((0.02, 1e-4, 1e-3))]
    state[2].square_()
    for t in state:
        t[n:] = 0
    sumsq = torch.empty(1, dtype=F64, device=CUDA)
    z.zero1_shard_grad_sumsq(plan, 0, M, grads, hp, sumsq)
    limit = 0.25 * sumsq.item() ** 0.5
    want, p = [torch.empty_like(t) for t in state], blank(n)
    z.zero1_step_clipped(plan, 0, M, grads, *state, p, hp, sumsq, limit, out=want)
    for mask in range(8):
        mine, q = [t.clone() for t in state], blank(n)
        out = [mine[k] if mask >> k & 1 else torch.empty_like(mine[k]) for k in range(3)]
        z.zero1_step_clipped(plan, 0, M, grads, *mine, q, hp, sumsq, limit, out=out)
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(p, q)
        assert all(torch.equal(a, b) for k, (a, b) in enumerate(zip(mine, state)) if not mask >> k & 1)
