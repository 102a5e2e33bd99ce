"""Layer norm, gated feed-forward block, weight gradient and clipping as programs
use them at the edges: captured and replayed, on two streams at once, again and
again with the same bits, with the caller's workspace, and over contractions that
are summed in several runs."""
import pytest
import torch

import ffn_reference as ref
import zero_sharded_mixed_zero1_gb300 as z

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def normal(*shape, std=1.0, seed=0, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


class Chain:
    """norm, feed-forward, its gradients, norm's gradients, clipping: one after the
    other on whatever stream is current."""

    def __init__(self, T, D, F, seed=0):
        e = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
        self.x, self.w, self.b = normal(T, D, seed=seed), normal(D, std=0.1, seed=seed + 1), normal(D, std=0.1, seed=seed + 2)
        self.wg, self.wu = normal(F, D, std=D ** -0.5, seed=seed + 3), normal(F, D, std=D ** -0.5, seed=seed + 4)
        self.da0 = normal(T, F, std=1e-3, seed=seed + 5)
        self.h, self.dh, self.dx = e(T, D), e(T, D), e(T, D)
        self.a, self.dg, self.du = e(T, F), e(T, F), e(T, F)
        self.mean, self.rstd = e(T, dtype=F32), e(T, dtype=F32)
        self.r8 = z.new_checkpoint(T, D, "cuda")
        self.grads = [e(F, D), e(F, D, dtype=F32), e(D), e(D)]
        self.clipped = [torch.zeros_like(t) for t in self.grads]
        self.sumsq, self.norms, self.norm = e(1, dtype=F64), e(4, dtype=F32), e(1, dtype=F32)

    def run(self):
        cfg = z.LayerNorm()
        z.zero1_layer_norm_forward(cfg, self.x, self.h, self.mean, self.rstd, w=self.w, b=self.b, r8=self.r8)
        z.zero1_gated_ffn_forward(self.h, self.wg, self.wu, self.a, act="gelu")
        z.zero1_gated_ffn_backward(self.da0, self.h, self.wg, self.wu, self.dg, self.du, a=self.a, act="gelu")
        z.zero1_gated_ffn_input_grad(self.dg, self.du, self.wg, self.wu, self.dh)
        z.zero1_weight_grad_bf16(self.dg, self.h, self.grads[0])
        z.zero1_weight_grad_bf16(self.du, self.h, self.grads[1])
        z.zero1_layer_norm_backward(cfg, self.dh, None, self.r8, self.mean, self.rstd, self.dx, w=self.w, dw=self.grads[2],
                                    db=self.grads[3])
        z.zero1_grad_sumsq(self.grads, self.sumsq, norms=self.norms)
        z.zero1_grad_clip(self.grads, self.sumsq, 1e-4, outs=self.clipped, norm=self.norm)

    def results(self):
        return [self.h, self.a, self.dg, self.du, self.dh, self.dx, self.mean, self.rstd, *self.grads, *self.clipped, self.sumsq,
                self.norms, self.norm]

    def clear(self):
        for t in self.results():
            t.zero_()


SIZES = [(200, 256, 512), (77, 133, 251), (9, 1024, 3000), (3000, 64, 96)]


@pytest.mark.parametrize("T,D,F", SIZES)
def test_the_same_bits_again_captured_and_replayed(T, D, F):
    c = Chain(T, D, F)
    c.run()
    want = [t.clone() for t in c.results()]
    for _ in range(3):
        c.clear()
        c.run()
        assert all(torch.equal(a, b) for a, b in zip(c.results(), want))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        c.run()
    for _ in range(3):
        c.clear()
        torch.cuda.synchronize()
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(c.results(), want))
    assert z.zero1_device_status() == 0


def test_two_streams_at_once():
    chains = [Chain(*SIZES[k], seed=10 * k) for k in (0, 1)]
    for c in chains:
        c.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.results()] for c in chains]
    streams = [torch.cuda.Stream() for _ in chains]
    for c in chains:
        c.clear()
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st in zip(chains, streams):
            with torch.cuda.stream(st):
                c.run()
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        assert all(torch.equal(a, b) for a, b in zip(c.results(), w))


def test_a_stream_argument_is_the_stream_that_is_used():
    """The call waits for what was enqueued on that stream, workspace and all."""
    T, D, F = 300, 200, 333
    h, wg, wu = normal(T, D), normal(F, D, std=0.05, seed=1), normal(F, D, std=0.05, seed=2)
    a, b = (torch.zeros(T, F, dtype=BF16, device="cuda") for _ in range(2))
    late = torch.zeros_like(h)
    torch.cuda.synchronize()
    z.zero1_gated_ffn_forward(h, wg, wu, a)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        late.copy_(h)
    z.zero1_gated_ffn_forward(late, wg, wu, b, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,D,F", [(200, 256, 512), (77, 133, 251), (9, 4096, 3000)])
def test_the_callers_workspace(T, D, F):
    """As many bytes as the query says, none behind them touched, one fewer refused."""
    c = Chain(T, D, F)
    c.run()
    want = [t.clone() for t in (c.a, c.dg, c.du, c.dh, c.grads[0], c.grads[1])]
    calls = [
        (z.zero1_gated_ffn_workspace("forward", T, c.wg, c.wu, h=c.h),
         lambda ws: z.zero1_gated_ffn_forward(c.h, c.wg, c.wu, c.a, act="gelu", workspace=ws)),
        (z.zero1_gated_ffn_workspace("backward", T, c.wg, c.wu, h=c.h),
         lambda ws: z.zero1_gated_ffn_backward(c.da0, c.h, c.wg, c.wu, c.dg, c.du, act="gelu", workspace=ws)),
        (z.zero1_gated_ffn_workspace("input_grad", T, c.wg, c.wu, dg=c.dg, du=c.du),
         lambda ws: z.zero1_gated_ffn_input_grad(c.dg, c.du, c.wg, c.wu, c.dh, workspace=ws)),
        (z.zero1_weight_grad_bf16_workspace(c.dg, c.h, BF16), lambda ws: z.zero1_weight_grad_bf16(c.dg, c.h, c.grads[0], workspace=ws)),
        (z.zero1_weight_grad_bf16_workspace(c.du, c.h, F32), lambda ws: z.zero1_weight_grad_bf16(c.du, c.h, c.grads[1], workspace=ws)),
        (z.zero1_layer_norm_workspace(T, D),
         lambda ws: z.zero1_layer_norm_backward(z.LayerNorm(), c.dh, None, c.r8, c.mean, c.rstd, c.dx, w=c.w, dw=c.grads[2], workspace=ws)),
        (z.zero1_grad_sumsq_workspace(c.grads), lambda ws: z.zero1_grad_sumsq(c.grads, c.sumsq, workspace=ws)),
    ]
    for nbytes, call in calls:
        flat = torch.full((nbytes + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        if nbytes:
            with pytest.raises(z.Zero1Error):
                call(flat[:nbytes - 1])
        call(flat[:nbytes])
        torch.cuda.synchronize()
        assert bool((flat[nbytes:] == 0xA5).all())
    assert all(torch.equal(a, b) for a, b in zip((c.a, c.dg, c.du, c.dh, c.grads[0], c.grads[1]), want))


@pytest.mark.parametrize("accumulate", [False, True])
def test_bf16_weight_gradients_of_several_runs(accumulate):
    """More than 131072 rows in whole tiles: the accumulator is emptied on the way."""
    T, N, K = 140_000, 2304, 2304
    dy, x = normal(T, N, std=1e-3, seed=1), normal(T, K, seed=2)
    dw = normal(N, K, std=1e-1, seed=3)
    start = dw.clone()
    z.zero1_weight_grad_bf16(dy, x, dw, accumulate=accumulate)
    rows = torch.tensor([0, 1, 255, 256, 1000, 2048, 2303], device="cuda")
    want = ref.weight_grad(dy[:, rows].contiguous(), x, BF16, start[rows] if accumulate else None)
    ref.check(dw[rows], want, "dw")


def test_offsets_beyond_32_bits():
    """Rows so far apart that element offsets leave 32 bits."""
    T, D, F = 5, 64, 128
    ld = (1 << 30) + 8
    flat = torch.empty(4 * ld + 256, dtype=BF16, device="cuda")  # 8.6 GB
    h = flat.as_strided((T, D), (ld, 1))
    h.copy_(normal(T, D))
    a = flat.as_strided((T, F), (ld, 1), 64)
    wg, wu = normal(F, D, std=0.1, seed=1), normal(F, D, std=0.1, seed=2)
    near_h, near_a = h.contiguous(), torch.empty(T, F, dtype=BF16, device="cuda")
    z.zero1_gated_ffn_forward(near_h, wg, wu, near_a)
    z.zero1_gated_ffn_forward(h, wg, wu, a)
    assert torch.equal(a, near_a)
    out, mean, rstd = flat.as_strided((T, D), (ld, 1), 192), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    near_out = torch.empty(T, D, dtype=BF16, device="cuda")
    z.zero1_layer_norm_forward(z.LayerNorm(), h, out, mean, rstd)
    z.zero1_layer_norm_forward(z.LayerNorm(), near_h, near_out, mean, rstd)
    assert torch.equal(out, near_out)
    # and one tensor of more than 2^32 elements in a list
    big = flat[:(1 << 32) + 5]
    big.zero_()
    big[-1], big[1 << 31], big[0] = 3.0, 4.0, 12.0
    sumsq = torch.empty(1, dtype=F64, device="cuda")
    z.zero1_grad_sumsq([big], sumsq)
    assert sumsq.item() == 169.0
    z.zero1_grad_clip([big], sumsq, 6.5)
    assert (big[-1].item(), big[1 << 31].item(), big[0].item()) == (1.5, 2.0, 6.0)


def test_pinned_host_memory():
    """Gradients and a residual stream in pinned host memory are read and written
    where they are; the feed-forward block, which is fed by copies of boxes, refuses
    them."""
    t = [normal(5001, seed=1).cpu().pin_memory(), normal(333, seed=2, dtype=F32).cpu().pin_memory(), normal(4096, seed=3)]
    near = [x.cuda() for x in t]
    a, b = (torch.empty(1, dtype=F64, device="cuda") for _ in range(2))
    z.zero1_grad_sumsq(t, a)
    z.zero1_grad_sumsq(near, b)
    assert torch.equal(a, b)
    z.zero1_grad_clip(t, a, 1.0)
    z.zero1_grad_clip(near, b, 1.0)
    torch.cuda.synchronize()
    assert all(torch.equal(x.cuda(), y) for x, y in zip(t, near))

    x = normal(40, 200, seed=4)
    far, out = x.cpu().pin_memory(), torch.empty(40, 200, dtype=BF16).pin_memory()
    h, stats = torch.empty_like(x), [torch.empty(40, device="cuda") for _ in range(2)]
    z.zero1_layer_norm_forward(z.LayerNorm(), x, h, *stats)
    z.zero1_layer_norm_forward(z.LayerNorm(), far, out, *stats)
    torch.cuda.synchronize()
    assert torch.equal(out.cuda(), h)

    wg, wu, act = normal(64, 200, seed=5), normal(64, 200, seed=6), torch.empty(40, 64, dtype=BF16, device="cuda")
    with pytest.raises(z.Zero1Error, match="device memory"):
        z.zero1_gated_ffn_forward(far, wg, wu, act)
    with pytest.raises(z.Zero1Error, match="device memory"):
        z.zero1_weight_grad_bf16(x, far, torch.empty(200, 200, dtype=BF16, device="cuda"))


def test_two_host_threads():
    """Calls from two threads at once, each on its own stream, give what they give alone."""
    import threading
    chains = [Chain(*SIZES[k], seed=10 * k) for k in (1, 2)]
    for c in chains:
        c.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.results()] for c in chains]
    wrong = []

    def work(k):
        try:
            torch.cuda.set_device(0)
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    chains[k].run()
        except Exception as e:  # noqa: BLE001
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(k,)) for k in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong
    for c, w in zip(chains, want):
        assert all(torch.equal(a, b) for a, b in zip(c.results(), w))
