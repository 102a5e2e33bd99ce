"""Layer norm, gated feed-forward block, weight gradient and clipping: outputs are
blanked before each call, so that one that writes nothing, or only a part, is seen."""
import threading

import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
from test_gpu_training_edges import SIZES, Chain

pytestmark = pytest.mark.gpu
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("T,D,F", [(200, 256, 512), (77, 133, 251), (9, 4096, 3000)])
def test_each_call_with_the_callers_workspace(T, D, F):
    c = Chain(T, D, F)
    c.run()
    torch.cuda.synchronize()
    dws = [torch.zeros_like(c.grads[2]) for _ in range(2)]
    z.zero1_layer_norm_backward(z.LayerNorm(), c.dh, None, c.r8, c.mean, c.rstd, c.dx, w=c.w, dw=dws[0], db=dws[1])
    assert same(dws[0], c.grads[2]) and same(dws[1], c.grads[3])
    calls = [
        (z.zero1_gated_ffn_workspace("forward", T, c.wg, c.wu, h=c.h), [c.a],
         lambda ws: z.zero1_gated_ffn_forward(c.h, c.wg, c.wu, c.a, act="gelu", workspace=ws)),
        (z.zero1_gated_ffn_workspace("backward", T, c.wg, c.wu, h=c.h), [c.dg, c.du, c.a],
         lambda ws: z.zero1_gated_ffn_backward(c.da0, c.h, c.wg, c.wu, c.dg, c.du, a=c.a, act="gelu", workspace=ws)),
        (z.zero1_gated_ffn_workspace("backward", T, c.wg, c.wu, h=c.h), [c.dg, c.du],
         lambda ws: z.zero1_gated_ffn_backward(c.da0, c.h, c.wg, c.wu, c.dg, c.du, act="gelu", workspace=ws)),
        (z.zero1_gated_ffn_workspace("input_grad", T, c.wg, c.wu, dg=c.dg, du=c.du), [c.dh],
         lambda ws: z.zero1_gated_ffn_input_grad(c.dg, c.du, c.wg, c.wu, c.dh, workspace=ws)),
        (z.zero1_weight_grad_bf16_workspace(c.dg, c.h, BF16), [c.grads[0]],
         lambda ws: z.zero1_weight_grad_bf16(c.dg, c.h, c.grads[0], workspace=ws)),
        (z.zero1_weight_grad_bf16_workspace(c.du, c.h, F32), [c.grads[1]],
         lambda ws: z.zero1_weight_grad_bf16(c.du, c.h, c.grads[1], workspace=ws)),
        (z.zero1_layer_norm_workspace(T, D), [c.dx, c.grads[2], c.grads[3]],
         lambda ws: z.zero1_layer_norm_backward(z.LayerNorm(), c.dh, None, c.r8, c.mean, c.rstd, c.dx, w=c.w, dw=c.grads[2],
                                                db=c.grads[3], workspace=ws)),
        (z.zero1_layer_norm_workspace(T, D), [c.dx, c.grads[3]],
         lambda ws: z.zero1_layer_norm_backward(z.LayerNorm(), c.dh, None, c.r8, c.mean, c.rstd, c.dx, w=c.w, db=c.grads[3], workspace=ws)),
        (z.zero1_grad_sumsq_workspace(c.grads), [c.sumsq, c.norms],
         lambda ws: z.zero1_grad_sumsq(c.grads, c.sumsq, norms=c.norms, workspace=ws)),
    ]
    for k, (nbytes, outs, call) in enumerate(calls):
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(float("nan"))
        call(torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want)), k


def test_two_host_threads_from_blank_results():
    chains = [Chain(*SIZES[k], seed=10 * k) for k in (1, 2)]
    for c in chains:
        c.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.results()] for c in chains]
    for c in chains:
        for t in c.results():
            t.fill_(float("nan"))
    torch.cuda.synchronize()
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
        assert all(same(a, b) for a, b in zip(c.results(), w))
    assert z.zero1_device_status() == 0


def test_two_graphs_replayed_at_once():
    """Each captured call has scratch memory of its own: two graphs may run at one time."""
    chains = [Chain(*SIZES[k], seed=10 * k) for k in (1, 2)]
    graphs, streams = [torch.cuda.CUDAGraph() for _ in chains], [torch.cuda.Stream() for _ in chains]
    for c in chains:
        c.run()
    torch.cuda.synchronize()
    want = [[t.clone() for t in c.results()] for c in chains]
    for c, g, st in zip(chains, graphs, streams):
        with torch.cuda.graph(g, stream=st):
            c.run()
    for c in chains:
        for t in c.results():
            t.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c, w in zip(chains, want):
        assert all(same(a, b) for a, b in zip(c.results(), w))
    assert z.zero1_device_status() == 0
