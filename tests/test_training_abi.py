"""The refusals of layer norm, gated feed-forward block, gradient norm and
clipping, without a GPU: every invalid argument is turned into an error code with a
reason before anything is launched.  Pointers here are numbers that nothing
dereferences."""
import ctypes
import struct

import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
from zero_sharded_mixed_zero1_gb300 import block as zb
from zero_sharded_mixed_zero1_gb300 import build as zbuild
from zero_sharded_mixed_zero1_gb300 import clip as zc
from zero_sharded_mixed_zero1_gb300 import ffn as zf
from zero_sharded_mixed_zero1_gb300 import layer_norm as zl

OK, EINVAL, EALIGN, ERANGE, ECUDA = 0, -1, -2, -3, -4
BF16, F32 = 0, 1
BASE = 1 << 32


def at(k, off=0):
    """Distinct 'buffers' 64 MiB apart."""
    return BASE + (k << 26) + off


@pytest.fixture(scope="module")
def lib():
    zbuild.build()
    zf._lib(), zl._lib()
    return zc._lib()


def reason(lib):
    return lib.zero1_last_error().decode()


def refused(lib, rc, code):
    assert rc == code, reason(lib)
    assert reason(lib)


def test_struct_sizes_are_the_headers(lib):
    assert (zl._CFG.size, zl._FWD.size, zl._BWD.size, zf._FFN.size) == (48, 104, 128, 160)


# ---------------------------------------------------------------- layer norm --

ROWS, COLS = 100, 200


def cfg(**kw):
    v = dict(rows=ROWS, cols=COLS, eps=1e-5, scale=1.0, act=BF16, res=BF16, param=BF16, grad=F32, accumulate=0)
    v.update(kw)
    return zl._CFG.pack(*v.values())


def fwd(**kw):
    v = dict(x=at(1), y=at(2), w=at(3), b=at(4), r=at(5), h=at(6), mean=at(7), rstd=at(8), r8=0, ld_x=COLS, ld_y=COLS, ld_r=COLS,
             ld_h=COLS)
    v.update(kw)
    return zl._FWD.pack(*v.values())


def bwd(**kw):
    v = dict(dh=at(1), dr=at(2), r=at(3), w=at(4), mean=at(5), rstd=at(6), r8=0, dx=at(7), dy=at(8), dw=at(9), db=at(10),
             ld_dh=COLS, ld_dr=COLS, ld_r=COLS, ld_dx=COLS, ld_dy=COLS)
    v.update(kw)
    return zl._BWD.pack(*v.values())


def ckpt(rows=ROWS, cols=COLS):
    return ctypes.create_string_buffer(zb._CKPT.pack(at(20), at(21), 256, 128, rows, cols), zb._CKPT.size)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL), (dict(cols=16385), ERANGE), (dict(rows=1 << 41), ERANGE),
    (dict(eps=0.0), EINVAL), (dict(eps=float("inf")), EINVAL), (dict(scale=float("nan")), EINVAL), (dict(act=2), EINVAL),
    (dict(res=-1), EINVAL), (dict(param=7), EINVAL), (dict(grad=3), EINVAL), (dict(act=F32), EINVAL),
])
def test_layer_norm_refuses_bad_configurations(lib, change, code):
    n = ctypes.c_int64()
    refused(lib, lib.zero1_layer_norm_forward(cfg(**change), fwd(), None), code)
    refused(lib, lib.zero1_layer_norm_backward(cfg(**change), bwd(), at(30), 1 << 30, None), code)
    refused(lib, lib.zero1_layer_norm_workspace(cfg(**change), ctypes.addressof(n)), code)


@pytest.mark.parametrize("change,code", [
    (dict(x=0), EINVAL), (dict(h=0), EINVAL), (dict(mean=0), EINVAL), (dict(rstd=0), EINVAL), (dict(y=0), EINVAL),
    (dict(r=0), EINVAL), (dict(x=at(1, 1)), EALIGN), (dict(w=at(3, 1)), EALIGN), (dict(rstd=at(8, 2)), EALIGN),
    (dict(ld_h=COLS - 1), EINVAL), (dict(ld_r=COLS - 1), EINVAL), (dict(ld_x=-1), EINVAL), (dict(ld_y=1 << 60), ERANGE),
    (dict(h=at(1)), EINVAL), (dict(r=at(2)), EINVAL), (dict(r=at(1, 16)), EINVAL), (dict(r=at(1), ld_r=COLS + 8), EINVAL),
    (dict(rstd=at(7)), EINVAL), (dict(h=at(3)), EINVAL), (dict(h=at(5, 64)), EINVAL),
])
def test_layer_norm_forward_refusals(lib, change, code):
    refused(lib, lib.zero1_layer_norm_forward(cfg(), fwd(**change), None), code)


@pytest.mark.parametrize("change,code", [
    (dict(dh=0), EINVAL), (dict(r=0), EINVAL), (dict(mean=0), EINVAL), (dict(rstd=0), EINVAL), (dict(dx=0), EINVAL),
    (dict(dh=at(1, 1)), EALIGN), (dict(dw=at(9, 2)), EALIGN), (dict(db=at(10, 1)), EALIGN), (dict(w=at(4, 1)), EALIGN),
    (dict(ld_dx=COLS - 1), EINVAL), (dict(ld_dh=-1), EINVAL), (dict(dx=at(1)), EINVAL), (dict(dx=at(2, 2)), EINVAL),
    (dict(dy=at(2)), EINVAL), (dict(dw=at(10)), EINVAL), (dict(dx=at(3)), EINVAL), (dict(dw=at(6)), EINVAL), (dict(db=at(30)), EINVAL),
])
def test_layer_norm_backward_refusals(lib, change, code):
    refused(lib, lib.zero1_layer_norm_backward(cfg(), bwd(**change), at(30), 1 << 20, None), code)


def test_layer_norm_checkpoint_refusals(lib):
    other, k = ckpt(rows=99), ckpt()
    refused(lib, lib.zero1_layer_norm_forward(cfg(), fwd(r8=ctypes.addressof(other)), None), EINVAL)
    assert "99 x 200" in reason(lib)
    refused(lib, lib.zero1_layer_norm_forward(cfg(), fwd(r8=ctypes.addressof(k), h=at(20)), None), EINVAL)
    refused(lib, lib.zero1_layer_norm_backward(cfg(), bwd(r8=ctypes.addressof(k)), at(30), 1 << 20, None), EINVAL)  # both
    refused(lib, lib.zero1_layer_norm_backward(cfg(), bwd(r=0, r8=ctypes.addressof(other)), at(30), 1 << 20, None), EINVAL)


def test_layer_norm_without_rows(lib):
    assert lib.zero1_layer_norm_forward(cfg(rows=0), fwd(x=0, h=0, mean=0, rstd=0, y=0, r=0), None) == OK


# --------------------------------------------------------------- feed-forward --

T, D, F = 100, 200, 300


def ffn(**kw):
    v = dict(rows=T, d=D, f=F, h=at(1), w_gate=at(2), w_up=at(3), da=at(4), a=at(5), dg=at(6), du=at(7), dh=at(8), ld_h=D,
             ld_w_gate=D, ld_w_up=D, ld_da=F, ld_a=F, ld_dg=F, ld_du=F, ld_dh=D, act=0)
    v.update(kw)
    return zf._FFN.pack(*v.values())


def calls(lib):
    return lib.zero1_gated_ffn_forward, lib.zero1_gated_ffn_backward, lib.zero1_gated_ffn_input_grad


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), EINVAL), (dict(d=0), EINVAL), (dict(f=0), EINVAL), (dict(act=2), EINVAL), (dict(act=-1), EINVAL),
    (dict(rows=1 << 31), ERANGE), (dict(d=1 << 30), ERANGE), (dict(f=1 << 30), ERANGE),
])
def test_gated_ffn_refuses_bad_sizes(lib, change, code):
    n = ctypes.c_int64()
    for k, call in enumerate(calls(lib)):
        refused(lib, call(ffn(**change), at(30), 1 << 30, None), code)
        refused(lib, lib.zero1_gated_ffn_workspace(ffn(**change), k, ctypes.addressof(n)), code)
        refused(lib, call(None, at(30), 1 << 30, None), EINVAL)
    refused(lib, lib.zero1_gated_ffn_workspace(ffn(), 3, ctypes.addressof(n)), EINVAL)
    refused(lib, lib.zero1_gated_ffn_workspace(ffn(), 0, None), EINVAL)


NEEDED = [("h", "w_gate", "w_up", "a"), ("h", "w_gate", "w_up", "da", "dg", "du"), ("dg", "du", "w_gate", "w_up", "dh")]


@pytest.mark.parametrize("kind", [0, 1, 2])
def test_gated_ffn_refuses_bad_matrices(lib, kind):
    call = calls(lib)[kind]
    outs = {0: ("a",), 1: ("dg", "du", "a"), 2: ("dh",)}[kind]
    where = dict(h=1, w_gate=2, w_up=3, da=4, a=5, dg=6, du=7, dh=8)
    for name in NEEDED[kind]:
        refused(lib, call(ffn(**{name: 0}), at(30), 1 << 30, None), EINVAL)
        refused(lib, call(ffn(**{name: at(where[name], 1)}), at(30), 1 << 30, None), EALIGN)
        refused(lib, call(ffn(**{"ld_" + name: -1}), at(30), 1 << 30, None), EINVAL)
        refused(lib, call(ffn(**{"ld_" + name: 1 << 61}), at(30), 1 << 30, None), ERANGE)
        for out in outs:
            if name != out and (name, out) != ("da", "dg"):
                refused(lib, call(ffn(**{out: at(where[name])}), at(30), 1 << 30, None), EINVAL)
    for out in outs:
        refused(lib, call(ffn(**{"ld_" + out: 10}), at(30), 1 << 30, None), EINVAL)
    if kind == 1:
        refused(lib, call(ffn(dg=at(4, 16)), at(30), 1 << 30, None), EINVAL)
        refused(lib, call(ffn(dg=at(4), ld_dg=F + 8), at(30), 1 << 30, None), EINVAL)


def test_gated_ffn_without_rows(lib):
    for call in calls(lib):
        assert call(ffn(rows=0, h=0, w_gate=0, da=0, a=0, dg=0, du=0, dh=0), None, 0, None) == OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU the accepted call would launch")
def test_gated_ffn_accepts_what_it_documents(lib):
    """These pass every check and then find no device."""
    fwd_, bwd_, grad = calls(lib)
    assert fwd_(ffn(da=0, dg=0, du=0, dh=0), None, 0, None) == ECUDA
    assert bwd_(ffn(a=0, dg=at(4), dh=0), None, 0, None) == ECUDA
    assert grad(ffn(h=0, da=0, a=0), None, 0, None) == ECUDA
    assert fwd_(ffn(ld_h=0, ld_w_gate=0), None, 0, None) == ECUDA  # rows that repeat


def wgrad(lib, **kw):
    v = dict(dy=at(1), ld_dy=F, n=F, x=at(2), ld_x=D, k=D, rows=T, dw=at(3), ld_dw=D, dtype=F32, accumulate=0, ws=at(30),
             bytes=1 << 30)
    v.update(kw)
    return lib.zero1_weight_grad_bf16(*v.values(), None)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), EINVAL), (dict(n=0), EINVAL), (dict(k=0), EINVAL), (dict(dtype=2), EINVAL), (dict(dy=0), EINVAL),
    (dict(x=0), EINVAL), (dict(dw=0), EINVAL), (dict(dy=at(1, 1)), EALIGN), (dict(dw=at(3, 2)), EALIGN), (dict(ld_dw=D - 1), EINVAL),
    (dict(ld_x=-1), EINVAL), (dict(dw=at(1)), EINVAL), (dict(dw=at(2, 64)), EINVAL), (dict(ld_dy=1 << 61), ERANGE),
])
def test_weight_grad_refusals(lib, change, code):
    refused(lib, wgrad(lib, **change), code)


# ------------------------------------------------------------ norm, clipping --

def table(*rows):
    return b"".join(struct.pack("=Qqii", *r) for r in rows)


GOOD = [(at(1), 1000, BF16, 0), (at(2), 77, F32, 0), (0, 0, BF16, 0)]


@pytest.mark.parametrize("row,code", [
    ((0, 5, BF16, 0), EINVAL), ((at(1), -1, BF16, 0), EINVAL), ((at(1), 5, 2, 0), EINVAL), ((at(1, 1), 5, BF16, 0), EALIGN),
    ((at(1, 2), 5, F32, 0), EALIGN), ((at(1), 1 << 41, BF16, 0), ERANGE),
])
def test_lists_refuse_bad_tensors(lib, row, code):
    n, t = ctypes.c_int64(), table(GOOD[1], row)
    refused(lib, lib.zero1_grad_sumsq_workspace(t, 2, ctypes.addressof(n)), code)
    refused(lib, lib.zero1_grad_sumsq(t, 2, at(10), None, 0, at(11), 1 << 20, None), code)
    refused(lib, lib.zero1_grad_clip(t, None, 2, at(10), 1.0, None, None), code)
    refused(lib, lib.zero1_grad_clip(table(GOOD[1], GOOD[0]), t, 2, at(10), 1.0, None, None), code)


def test_lists_refuse_what_else_is_wrong(lib):
    t, two = table(*GOOD), table(GOOD[0], GOOD[0])
    refused(lib, lib.zero1_grad_sumsq(None, 2, at(10), None, 0, at(11), 1 << 20, None), EINVAL)
    refused(lib, lib.zero1_grad_sumsq(t, -1, at(10), None, 0, at(11), 1 << 20, None), EINVAL)
    refused(lib, lib.zero1_grad_sumsq(t, 3, None, None, 0, at(11), 1 << 20, None), EINVAL)
    refused(lib, lib.zero1_grad_sumsq(t, 3, at(10, 4), None, 0, at(11), 1 << 20, None), EALIGN)
    refused(lib, lib.zero1_grad_sumsq(t, 3, at(10), at(12, 2), 0, at(11), 1 << 20, None), EALIGN)
    for place in (dict(sumsq=at(1, 16)), dict(norms=at(2)), dict(norms=at(10)), dict(ws=at(1)), dict(ws=at(10))):
        v = dict(sumsq=at(10), norms=at(12), accumulate=0, ws=at(11))
        v.update(place)
        refused(lib, lib.zero1_grad_sumsq(t, 3, *v.values(), 1 << 20, None), EINVAL)
    for limit in (0.0, -1.0, float("nan"), float("inf")):
        refused(lib, lib.zero1_grad_clip(t, None, 3, at(10), limit, None, None), EINVAL)
    refused(lib, lib.zero1_grad_clip(t, None, 3, None, 1.0, None, None), EINVAL)
    refused(lib, lib.zero1_grad_clip(two, None, 2, at(10), 1.0, None, None), EINVAL)                   # scaled twice
    refused(lib, lib.zero1_grad_clip(t, None, 3, at(1, 8), 1.0, None, None), EINVAL)                   # sumsq inside a tensor
    refused(lib, lib.zero1_grad_clip(t, None, 3, at(10), 1.0, at(10), None), EINVAL)
    refused(lib, lib.zero1_grad_clip(t, table(GOOD[1], GOOD[0], GOOD[2]), 3, at(10), 1.0, None, None), EINVAL)  # other sizes
    # outputs on one another, and on another tensor's input
    refused(lib, lib.zero1_grad_clip(table((at(1), 8, BF16, 0), (at(2), 8, BF16, 0)), table((at(5), 8, BF16, 0), (at(5, 8), 8, BF16, 0)), 2,
                                     at(10), 1.0, None, None), EINVAL)
    refused(lib, lib.zero1_grad_clip(table((at(1), 8, BF16, 0), (at(2), 8, BF16, 0)), table((at(2), 8, BF16, 0), (at(5), 8, BF16, 0)), 2,
                                     at(10), 1.0, None, None), EINVAL)
    refused(lib, lib.zero1_grad_clip(table((at(1), 8, BF16, 0)), table((at(1, 2), 8, BF16, 0)), 1, at(10), 1.0, None, None), EINVAL)


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU the accepted call would launch")
def test_lists_accept_what_they_document(lib):
    t = table(*GOOD)
    assert lib.zero1_grad_sumsq(table(*GOOD, *GOOD), 6, at(10), None, 0, at(11), 1 << 20, None) == ECUDA  # tensors may repeat
    assert lib.zero1_grad_clip(t, None, 3, at(10), 1.0, at(12), None) == ECUDA
    assert lib.zero1_grad_clip(t, t, 3, at(10), 1.0, at(12), None) == ECUDA
    assert lib.zero1_grad_clip(t, table((at(5), 1000, BF16, 0), GOOD[1], GOOD[2]), 3, at(10), 1.0, None, None) == ECUDA


HP = z.AdamW(global_batch=64, step=3)


def shard(lib, plan=None, hp=HP, grads=None, **kw):
    plan = z.zero1_plan(1000, 2, 8) if plan is None else plan
    g = struct.pack("=2Q", at(1), at(2)) if grads is None else grads
    v = dict(begin=0, end=2, sumsq=at(10), sums=at(11), accumulate=0, ws=at(12), bytes=1 << 20)
    v.update(kw)
    return lib.zero1_shard_grad_sumsq(ctypes.byref(plan), v["begin"], v["end"], g, ctypes.byref(hp.c_struct()), v["sumsq"], v["sums"],
                                      v["accumulate"], v["ws"], v["bytes"], None)


@pytest.mark.parametrize("change,code", [
    (dict(begin=-1), EINVAL), (dict(end=3), EINVAL), (dict(begin=1, end=1), EINVAL), (dict(sumsq=None), EINVAL),
    (dict(sumsq=at(10, 4)), EALIGN), (dict(sums=at(11, 2)), EALIGN), (dict(sums=at(1)), EINVAL), (dict(sums=at(10)), EINVAL),
    (dict(ws=None), EINVAL), (dict(bytes=100), EINVAL), (dict(ws=at(12, 4)), EALIGN), (dict(ws=at(2)), EINVAL),
    (dict(grads=struct.pack("=2Q", at(1), 0)), EINVAL), (dict(grads=struct.pack("=2Q", at(1), at(2, 1))), EALIGN),
    (dict(hp=z.AdamW(global_batch=1)), EINVAL), (dict(hp=z.AdamW(global_batch=64, loss_scale=0.0)), EINVAL),
])
def test_shard_sumsq_refusals(lib, change, code):
    refused(lib, shard(lib, **change), code)


def step(lib, hp=HP, **kw):
    plan = z.zero1_plan(1000, 2, 8)
    v = dict(begin=0, end=2, grads=struct.pack("=2Q", at(1), at(2)), sums=None, w=at(3), m=at(4), v=at(5), wo=at(3), mo=at(4),
             vo=at(5), params=at(6), sumsq=at(7), max_norm=1.0, norm=at(8), flag=at(9))
    v.update(kw)
    return lib.zero1_step_clipped(ctypes.byref(plan), v["begin"], v["end"], v["grads"], v["sums"], v["w"], v["m"], v["v"], v["wo"], v["mo"],
                                  v["vo"], v["params"], ctypes.byref(hp.c_struct()), v["sumsq"], v["max_norm"], v["norm"], v["flag"], None)


@pytest.mark.parametrize("change,code", [
    (dict(end=3), EINVAL), (dict(grads=None), EINVAL), (dict(w=None), EINVAL), (dict(vo=None), EINVAL), (dict(params=None), EINVAL),
    (dict(sumsq=None), EINVAL), (dict(max_norm=0.0), EINVAL), (dict(max_norm=float("nan")), EINVAL),
    (dict(max_norm=float("inf")), EINVAL), (dict(w=at(3, 2)), EALIGN), (dict(mo=at(13, 1)), EALIGN), (dict(params=at(6, 1)), EALIGN),
    (dict(sumsq=at(7, 4)), EALIGN), (dict(sums=at(12, 1)), EALIGN), (dict(norm=at(8, 2)), EALIGN), (dict(flag=at(9, 1)), EALIGN),
    (dict(wo=at(4), mo=at(3)), EINVAL), (dict(wo=at(3, 16)), EINVAL), (dict(params=at(1)), EINVAL), (dict(params=at(3)), EINVAL),
    (dict(wo=at(2)), EINVAL), (dict(norm=at(7)), EINVAL), (dict(norm=at(6, 4)), EINVAL), (dict(flag=at(8)), EINVAL),
    (dict(sums=at(3)), EINVAL), (dict(hp=z.AdamW(global_batch=64, beta1=1.0)), EINVAL), (dict(hp=z.AdamW(global_batch=1)), EINVAL),
])
def test_clipped_step_refusals(lib, change, code):
    refused(lib, step(lib, **change), code)


# ------------------------------------------------------------- the binding --

def test_the_binding_refuses_host_tensors_and_wrong_types(lib):
    """(On a machine without a driver torch itself refuses to name the current
    device, with a RuntimeError.)"""
    x = torch.zeros(4, 8)
    wrong = (TypeError, ValueError, RuntimeError)
    for call in (lambda: z.zero1_grad_sumsq([x], torch.zeros(1, dtype=torch.float64)),
                 lambda: z.zero1_grad_sumsq([3], torch.zeros(1, dtype=torch.float64)),
                 lambda: z.zero1_grad_clip([x], torch.zeros(1, dtype=torch.float64), 1.0, outs=[]),
                 lambda: z.zero1_layer_norm_forward(z.LayerNorm(), x, x, torch.zeros(4), torch.zeros(4)),
                 lambda: z.zero1_layer_norm_forward(z.LayerNorm(), x.half(), x, torch.zeros(4), torch.zeros(4)),
                 lambda: z.zero1_gated_ffn_forward(x[0], x, x, x),
                 lambda: z.zero1_gated_ffn_forward(x, x, x, x),
                 lambda: z.zero1_gated_ffn_forward(x, x, x, x, act="relu"),
                 lambda: z.zero1_gated_ffn_workspace("sideways", 4, x, x),
                 lambda: z.zero1_weight_grad_bf16(x, x, x)):
        with pytest.raises(wrong):
            call()
