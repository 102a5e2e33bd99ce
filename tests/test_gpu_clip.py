"""The global gradient norm and clipping on the GPU: lists of tensors against
float64, the clipped step bit for bit against the fused step where nothing is
scaled and against its own formula in fp32 where something is."""
import math

import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
# a sum of squares: at most 8 + 16 roundings to fp32 on the way into doubles, which add less than one more
SUMSQ = 25 * 2.0 ** -24


def dev(dtype, n=1):
    return torch.full((n,), float("nan"), dtype=dtype, device="cuda")


def normal(n, std, seed, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * std).to(dtype)


def lists(sizes, dtype, offset=0, std=1e-2):
    flat = normal(offset + sum(sizes), std, 1, dtype)
    return list(torch.split(flat[offset:], sizes))


SIZES = [[1], [8], [7, 0, 9], [100003], [5] * 700, [1 << 20, 3, 0, 17, 4096, 65537], [2048 * 8, 2048 * 8 + 5], [0, 0], []]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("k", range(len(SIZES)))
def test_norm_and_clip_of_lists(k, offset, dtype):
    t = lists(SIZES[k], dtype, offset)
    n = len(t)
    sumsq, norms, norm = dev(F64), dev(F32, max(n, 1)), dev(F32)
    z.zero1_grad_sumsq(t, sumsq, norms=norms)
    want = torch.tensor([x.double().square().sum().item() for x in t], dtype=F64)
    total = want.sum().item()
    assert abs(sumsq.item() - total) <= SUMSQ * total
    assert torch.allclose(norms[:n].cpu().double(), want.sqrt(), rtol=SUMSQ, atol=0)
    real = math.sqrt(sumsq.item())
    for ratio in (0.37, 2.0):
        limit = max(ratio * real, 1e-3)
        c = min(1.0, torch.tensor(limit, dtype=F32).item() / (real + 1e-6))
        c = torch.tensor(c, dtype=F64).float().item()
        ref = [(x.float() * c).to(dtype) for x in t]
        flat = torch.full((offset + sum(SIZES[k]) + 9,), 5.0, dtype=dtype, device="cuda")
        for shift in (offset, offset + 1):  # the same place within 16 bytes, and another
            flat.fill_(5.0)
            outs = list(torch.split(flat[shift:shift + sum(SIZES[k])], SIZES[k]))
            before = [x.clone() for x in t]
            z.zero1_grad_clip(t, sumsq, limit, outs=outs, norm=norm)
            for a, b, d, e in zip(outs, ref, t, before):
                assert torch.equal(a, b) and torch.equal(d, e)
            assert bool((flat[:shift] == 5).all()) and bool((flat[shift + sum(SIZES[k]):] == 5).all())
            assert abs(norm.item() - real) <= 2.0 ** -23 * real
        mine = [x.clone() for x in t]
        z.zero1_grad_clip(mine, sumsq, limit)
        for a, b in zip(mine, ref):
            assert torch.equal(a, b)


def test_types_may_differ_and_tensors_repeat():
    a, b = normal(1000, 1.0, 1, BF16), normal(333, 1.0, 2, F32).view(3, 111)
    sumsq = dev(F64)
    z.zero1_grad_sumsq([a, b, a], sumsq)
    want = 2 * a.double().square().sum().item() + b.double().square().sum().item()
    assert abs(sumsq.item() - want) <= SUMSQ * want
    z.zero1_grad_sumsq([b], sumsq, accumulate=True)
    want += b.double().square().sum().item()
    assert abs(sumsq.item() - want) <= SUMSQ * want
    with pytest.raises(z.Zero1Error):
        z.zero1_grad_clip([a, b, a], sumsq, 1.0)
    with pytest.raises(z.Zero1Error):
        z.zero1_grad_clip([a, b], sumsq, 1.0, outs=[a[:1000], a[:333 * 2].view(torch.float32)[:333].view(3, 111)])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e-20, 1e20, 1e30, 1e38])
@pytest.mark.parametrize("n", [1, 5, 8, 5000])
def test_sizes_whose_squares_leave_fp32(size, n, dtype):
    t = normal(n, size, 3, dtype)
    t = torch.where(torch.isfinite(t), t, torch.full_like(t, size))
    sumsq = dev(F64)
    z.zero1_grad_sumsq([t], sumsq)
    want = t.double().square().sum().item()
    assert abs(sumsq.item() - want) <= SUMSQ * want


def test_tiny_among_large_zero_and_subnormal():
    for values in ([0.0] * 64, [0.0, -0.0, 1e-40, 2e-45] * 16, [1e-25] * 32 + [1.0] * 32, [3e38] + [1e-38] * 63):
        t = torch.tensor(values, device="cuda")
        sumsq = dev(F64)
        z.zero1_grad_sumsq([t], sumsq)
        want = t.double().square().sum().item()
        assert abs(sumsq.item() - want) <= SUMSQ * want


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("at", [0, 3, 1000, 9999])
def test_gradients_that_are_not_finite_stay(bad, at):
    t = normal(10000, 1.0, 1, BF16)[1:]
    t[at - 1 if at else 0] = bad
    keep = t.clone()
    sumsq, norm = dev(F64), dev(F32)
    z.zero1_grad_sumsq([t], sumsq)
    assert not math.isfinite(sumsq.item())
    z.zero1_grad_clip([t], sumsq, 1e-3, norm=norm)
    assert torch.equal(t.view(torch.int16), keep.view(torch.int16)) and not math.isfinite(norm.item())


# ------------------------------------------------------------------ the step --

HP = z.AdamW(lr=1e-3, weight_decay=0.1, global_batch=64, loss_scale=128.0, step=7)


class Step:
    def __init__(self, n, M, align=1, offset=0, std=1.0):
        self.plan = z.zero1_plan(n, M, align)
        P = self.plan.padded_n
        self.n, self.M = n, M
        self.grads = [normal(offset + n, std, 10 + r, BF16)[offset:] for r in range(M)]
        f = [normal(offset + P, s, 50 + k, F32)[offset:] for k, s in enumerate((0.02, 1e-4, 1e-3))]
        self.master, self.m, self.v = f[0], f[1], f[2].square_()
        for t in f:
            t[n:] = 0
        self.params = torch.zeros(offset + n, dtype=BF16, device="cuda")[offset:]

    def copies(self):
        return [t.clone() for t in (self.master, self.m, self.v, self.params)]

    def gradient(self):
        s = self.grads[0].float()
        for g in self.grads[1:]:
            s = s + g.float()
        return s

    def sumsq(self, sums=None, begin=0, end=None, accumulate=False, into=None):
        q = dev(F64) if into is None else into
        end = self.M if end is None else end
        base, _, nv = self.plan.shard_range(begin, end)
        z.zero1_shard_grad_sumsq(self.plan, begin, end, [g[base:base + nv] for g in self.grads], HP, q, sums=sums, accumulate=accumulate)
        return q


STEPS = [(1, 1, 1), (5, 3, 8), (1000, 2, 128), (4099, 5, 1), (100003, 8, 8), (65536, 4, 128), (30011, 13, 1), (9000, 64, 4), (1 << 21, 1, 1)]


@pytest.mark.parametrize("offset", [0, 1, 8])
@pytest.mark.parametrize("n,M,align", STEPS)
def test_clipped_step(n, M, align, offset):
    s = Step(n, M, align, offset)
    inv = torch.tensor(1.0 / (HP.global_batch * HP.loss_scale), dtype=F64).float().item()
    g = s.gradient() * inv
    want = g.double().square().sum().item()
    sums = dev(F32, s.plan.padded_n)
    q = s.sumsq()
    assert abs(q.item() - want) <= SUMSQ * want
    assert abs(s.sumsq(sums=sums).item() - want) <= SUMSQ * want  # (where sums lies may change the order)
    assert torch.equal(s.sumsq(), q)
    assert torch.equal(sums[:n], s.gradient()) and bool((sums[n:] == 0).all())
    norm = math.sqrt(q.item())

    # nothing scaled: the fused step, bit for bit
    fused, clipped = s.copies(), s.copies()
    z.zero1_reduce_scatter_adamw_allgather(s.plan, 0, M, s.grads, *fused, HP)
    z.zero1_step_clipped(s.plan, 0, M, s.grads, *clipped, HP, q, 2 * norm + 1.0)
    for a, b in zip(fused, clipped):
        assert torch.equal(a, b)

    # scaled: AdamW on g * c in fp32, each operation rounded once
    limit = torch.tensor(norm * 0.3, dtype=F32).item()
    c = torch.tensor(limit / (norm + 1e-6), dtype=F64).float().item()
    f = z.AdamW(lr=HP.lr, weight_decay=HP.weight_decay, global_batch=M, step=HP.step)
    gc = torch.zeros(s.plan.padded_n, device="cuda")
    gc[:n] = g * c
    adam = s.copies()
    z.zero1_adamw_update(s.plan, 0, M, gc, *adam[:3], f)
    out = [torch.empty_like(t) for t in adam[:3]]
    before = s.copies()
    said, flag = dev(F32), torch.zeros(1, dtype=torch.int32, device="cuda")
    for kept in (None, sums):
        for to in (None, out):
            mine = s.copies()
            z.zero1_step_clipped(s.plan, 0, M, None if kept is not None else s.grads, *mine, HP, q, limit, sums=kept, out=to,
                                 norm=said, overflow_flag=flag)
            got = mine[:3] if to is None else out
            for a, b in zip(got, adam):
                assert torch.equal(a, b)
            if to is not None:
                for a, b in zip(mine[:3], before):
                    assert torch.equal(a, b)
            assert torch.equal(mine[3], adam[0][:n].to(BF16))
            assert abs(said.item() - norm) <= 2.0 ** -23 * norm and flag.item() == 0


def test_ranks_add_their_shards():
    """Each rank's shards on their own, sums added, then each rank's step: the whole step."""
    s = Step(10007, 4, 8)
    whole = s.sumsq()
    total = torch.zeros(1, dtype=F64, device="cuda")
    for k in range(4):
        s.sumsq(begin=k, end=k + 1, accumulate=True, into=total)
    assert abs(total.item() - whole.item()) <= 2 * SUMSQ * whole.item()
    limit = 0.5 * math.sqrt(total.item())
    one, parts = s.copies(), s.copies()
    z.zero1_step_clipped(s.plan, 0, 4, s.grads, *one, HP, total, limit)
    for k in range(4):
        base, L, nv = s.plan.shard_range(k, k + 1)
        w, m, v, p = parts
        z.zero1_step_clipped(s.plan, k, k + 1, [g[base:base + nv] for g in s.grads], w[base:base + L], m[base:base + L],
                             v[base:base + L], p[base:base + nv], HP, total, limit)
    for a, b in zip(one, parts):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_an_overflow_skips_the_clipped_step(bad, kept):
    s = Step(5001, 3, 8)
    s.grads[1][17] = bad
    sums = dev(F32, s.plan.padded_n) if kept else None
    q = s.sumsq(sums=sums)
    assert not math.isfinite(q.item())
    mine, before = s.copies(), s.copies()
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    z.zero1_step_clipped(s.plan, 0, 3, s.grads, *mine, HP, q, 1.0, sums=sums, overflow_flag=flag)
    for a, b in zip(mine, before):
        assert torch.equal(a, b)
    assert flag.item() == 1


def test_a_captured_step_on_another_stream():
    s = Step(70001, 4, 8)
    q, out = dev(F64), s.copies()
    st = torch.cuda.Stream()
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    limit = 0.25 * math.sqrt(s.sumsq().item())
    with torch.cuda.stream(st):
        def step():
            z.zero1_shard_grad_sumsq(s.plan, 0, 4, s.grads, HP, q, workspace=ws)
            z.zero1_step_clipped(s.plan, 0, 4, s.grads, s.master, s.m, s.v, out[3], HP, q, limit, out=out[:3])
            z.zero1_grad_sumsq(s.grads, q, accumulate=True, workspace=ws)
        step()
        st.synchronize()
        want = [t.clone() for t in out] + [q.clone()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
    for t in out:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out + [q], want):
        assert torch.equal(a, b)
