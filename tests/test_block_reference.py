"""The 64-bit formulas that the kernels are held to, checked without a GPU:
the gradients against central differences and against automatic
differentiation, the 8-bit code against a library cast."""
import pytest
import torch

import block_reference as ref


def problem(T, D, post, pre, gate, act):
    g = torch.Generator().manual_seed(T * 100 + D)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    shape = {None: None, "channel": (D,), "token": (T, 1), "full": (T, D)}[gate]
    return {"y": r(T, D), "x": r(T, D), "w_post": 1 + 0.1 * r(D) if post else None,
            "w_pre": 1 + 0.1 * r(D) if pre else None, "gate": None if shape is None else r(*shape)}


def loss_of(p, act, ch, cr):
    f = ref.forward(p["y"], p["x"], p["w_post"], p["w_pre"], p["gate"], act, 0.7, 1e-6)
    s = (f["r"] * cr).sum()
    return s if f["h"] is None else s + (f["h"] * ch).sum()


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("gate", [None, "channel", "token", "full"])
@pytest.mark.parametrize("act", ["linear", "sigmoid"])
def test_gradients_against_differences_and_autograd(post, pre, gate, act):
    T, D = 3, 5
    p = problem(T, D, post, pre, gate, act)
    g = torch.Generator().manual_seed(1)
    ch, cr = (torch.randn((T, D), generator=g, dtype=torch.float64) for _ in range(2))
    f = ref.forward(p["y"], p["x"], p["w_post"], p["w_pre"], p["gate"], act, 0.7, 1e-6)
    got = ref.backward(ch if pre else None, cr, f["yh"], f["rh"], f["rstd_post"], f["rstd_pre"], p["w_post"],
                       p["w_pre"], p["gate"], act, 0.7)
    names = {"y": "dy", "x": "dx", "w_post": "dw_post", "w_pre": "dw_pre", "gate": "dgate"}
    leaves = {k: t.clone().requires_grad_() for k, t in p.items() if t is not None}
    loss_of({k: leaves.get(k) for k in p}, act, ch, cr).backward()
    for k, t in p.items():
        if t is None:
            continue
        assert torch.allclose(got[names[k]], leaves[k].grad, rtol=1e-11, atol=1e-12), k
        flat, step = t.view(-1), 1e-6
        for j in range(flat.numel()):
            keep = flat[j].item()
            flat[j] = keep + step
            hi = loss_of(p, act, ch, cr)
            flat[j] = keep - step
            lo = loss_of(p, act, ch, cr)
            flat[j] = keep
            # central differences: truncation O(step^2), cancellation 1e-16 / step
            assert abs((hi - lo) / (2 * step) - got[names[k]].reshape(-1)[j]) < 1e-7, (k, j)


def test_pack_against_the_library_cast():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((50, 300), generator=g) * torch.exp(8 * torch.randn((50, 1), generator=g))
    codes, exps = ref.pack(x.double())
    v = torch.nn.functional.pad(x, (0, 84)).view(50, 3, 128)
    q = v * (2.0 ** (127 - exps.double())).float()[:, :, None]
    assert torch.equal(codes, q.to(torch.float8_e4m3fn).view(torch.uint8).view(50, 384))
    assert q.abs().amax() <= 448 and (q.abs().amax(dim=2) > 224).all()
    assert ((ref.values(codes, exps, 300) - x).abs() <= x.abs() * 2.0 ** -4 + 2.0 ** -10 *
            (2.0 ** (exps.double() - 127)).repeat_interleave(128, 1)[:, :300]).all()
