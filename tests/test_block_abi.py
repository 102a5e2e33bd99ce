"""The training-block operators' refusals, without a GPU: every invalid
argument is turned into an error code with a reason before anything is
launched.  Pointers here are numbers that nothing dereferences."""
import ctypes

import pytest
import torch

import zero_sharded_mixed_zero1_gb300 as z
from zero_sharded_mixed_zero1_gb300 import block as zb
from zero_sharded_mixed_zero1_gb300 import build as zbuild

OK, EINVAL, EALIGN, ERANGE, ECUDA = 0, -1, -2, -3, -4
BF16, F32 = 0, 1
BASE = 1 << 32


def at(k, off=0):
    """Distinct 'buffers' 64 MiB apart."""
    return BASE + (k << 26) + off


@pytest.fixture(scope="module")
def lib():
    zbuild.build()
    return zb._lib()


def ckpt(rows=100, cols=200, codes=at(20), exps=at(21), ld_codes=256, ld_exps=128):
    return ctypes.create_string_buffer(zb._CKPT.pack(codes, exps, ld_codes, ld_exps, rows, cols), zb._CKPT.size)


def reason(lib):
    return lib.zero1_last_error().decode()


# --------------------------------------------------------------- checkpoints --

def test_struct_sizes_are_the_headers(lib):
    assert (zb._CKPT.size, zb._CFG.size, zb._FWD.size, zb._BWD.size) == (48, 56, 128, 192)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), EINVAL), (dict(cols=0), EINVAL), (dict(codes=0), EINVAL), (dict(exps=0), EINVAL),
    (dict(codes=at(20, 8)), EALIGN), (dict(exps=at(21, 4)), EALIGN), (dict(ld_codes=264), EALIGN),
    (dict(ld_codes=240), EINVAL), (dict(ld_exps=112), EINVAL), (dict(cols=257), EINVAL), (dict(rows=129), EINVAL),
    (dict(rows=1 << 41, ld_exps=1 << 41), ERANGE), (dict(exps=at(20, 256)), EINVAL),
])
def test_checkpoint_refusals(lib, change, code):
    k = ckpt(**change)
    for call in (lambda: lib.zero1_checkpoint_pack(at(1), 200, BF16, ctypes.addressof(k), None),
                 lambda: lib.zero1_checkpoint_unpack(ctypes.addressof(k), at(1), max(200, 257), BF16, None)):
        assert call() == code, reason(lib)
        assert reason(lib)


def test_pack_and_unpack_refuse_bad_matrices(lib):
    k = ckpt()
    a = ctypes.addressof(k)
    assert lib.zero1_checkpoint_pack(None, 200, BF16, a, None) == EINVAL
    assert lib.zero1_checkpoint_pack(at(1), -1, BF16, a, None) == EINVAL
    assert lib.zero1_checkpoint_pack(at(1), 200, 2, a, None) == EINVAL
    assert lib.zero1_checkpoint_pack(at(1, 1), 200, BF16, a, None) == EALIGN
    assert lib.zero1_checkpoint_pack(at(1, 2), 200, F32, a, None) == EALIGN
    assert lib.zero1_checkpoint_pack(at(1), 200, BF16, None, None) == EINVAL
    assert lib.zero1_checkpoint_pack(at(20, 512), 200, BF16, a, None) == EINVAL          # x inside the codes
    assert lib.zero1_checkpoint_unpack(a, at(1), 199, BF16, None) == EINVAL               # rows of out overlap
    assert lib.zero1_checkpoint_pack(at(1), 1 << 60, F32, a, None) == ERANGE
    empty = ckpt(rows=0, codes=0, exps=0)
    assert lib.zero1_checkpoint_pack(None, 0, BF16, ctypes.addressof(empty), None) == OK  # nothing to do


# --------------------------------------------------------------- block norms --

ROWS, COLS = 100, 200


def cfg(**kw):
    v = dict(rows=ROWS, cols=COLS, eps=1e-6, scale=1.0, act=BF16, res=BF16, param=BF16, gate=BF16, grad=F32, kind=0,
             gate_act=0, accumulate=0)
    v.update(kw)
    return zb._CFG.pack(*v.values())


def fwd(**kw):
    v = dict(y=at(1), x=at(2), w_post=at(3), w_pre=at(4), gate=0, r=at(5), h=at(6), rstd_post=at(7), rstd_pre=at(8), y8=0,
             r8=0, ld_y=COLS, ld_x=COLS, ld_gate=0, ld_r=COLS, ld_h=COLS)
    v.update(kw)
    return zb._FWD.pack(*v.values())


def bwd(**kw):
    v = dict(dh=at(1), dr=at(2), y=at(3), r=at(4), w_post=at(5), w_pre=at(6), gate=0, rstd_post=at(7), rstd_pre=at(8), y8=0,
             r8=0, dy=at(9), dx=at(10), dw_post=at(11), dw_pre=at(12), dgate=0, ld_dh=COLS, ld_dr=COLS, ld_y=COLS,
             ld_r=COLS, ld_gate=0, ld_dy=COLS, ld_dx=COLS, ld_dgate=0)
    v.update(kw)
    return zb._BWD.pack(*v.values())


BAD_CFG = [(dict(rows=-1), EINVAL), (dict(cols=0), EINVAL), (dict(cols=16385), ERANGE), (dict(rows=1 << 41), ERANGE),
           (dict(eps=0.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(scale=float("inf")), EINVAL),
           (dict(act=2), EINVAL), (dict(res=-1), EINVAL), (dict(param=7), EINVAL), (dict(gate=2), EINVAL),
           (dict(grad=3), EINVAL), (dict(act=F32), EINVAL), (dict(kind=4), EINVAL), (dict(gate_act=2), EINVAL),
           (dict(kind=1), EINVAL)]


@pytest.mark.parametrize("change,code", BAD_CFG)
def test_block_norm_refuses_bad_configurations(lib, change, code):
    n = ctypes.c_int64()
    assert lib.zero1_block_norm_forward(cfg(**change), fwd(), None) == code, reason(lib)
    assert lib.zero1_block_norm_backward(cfg(**change), bwd(), at(30), 1 << 30, None) == code, reason(lib)
    if change != dict(kind=1):
        assert lib.zero1_block_norm_workspace(cfg(**change), ctypes.addressof(n)) == code, reason(lib)


@pytest.mark.parametrize("change,code", [
    (dict(y=0), EINVAL), (dict(x=0), EINVAL), (dict(r=0), EINVAL), (dict(h=0), EINVAL), (dict(rstd_post=0), EINVAL),
    (dict(rstd_pre=0), EINVAL), (dict(w_post=0), EINVAL), (dict(w_pre=0), EINVAL), (dict(gate=at(9)), EINVAL),
    (dict(y=at(1, 1)), EALIGN), (dict(w_pre=at(4, 1)), EALIGN), (dict(rstd_pre=at(8, 2)), EALIGN),
    (dict(ld_r=COLS - 1), EINVAL), (dict(ld_y=-1), EINVAL), (dict(r=at(1)), EINVAL), (dict(h=at(5)), EINVAL),
    (dict(r=at(2, 16)), EINVAL), (dict(rstd_pre=at(7)), EINVAL), (dict(h=at(3)), EINVAL),
])
def test_forward_refusals(lib, change, code):
    assert lib.zero1_block_norm_forward(cfg(), fwd(**change), None) == code, reason(lib)


def test_forward_checkpoint_refusals(lib):
    other = ckpt(rows=99)
    assert lib.zero1_block_norm_forward(cfg(), fwd(y8=ctypes.addressof(other)), None) == EINVAL
    assert "99 x 200" in reason(lib)
    k = ckpt()
    assert lib.zero1_block_norm_forward(cfg(), fwd(y8=ctypes.addressof(k), r8=ctypes.addressof(k)), None) == EINVAL
    assert lib.zero1_block_norm_forward(cfg(), fwd(w_pre=0, h=0, rstd_pre=0, r8=ctypes.addressof(k)), None) == EINVAL


@pytest.mark.skipif(torch.cuda.is_available(), reason="with a GPU the accepted call would launch")
def test_interleaved_columns_of_one_matrix_do_not_overlap(lib):
    """r and h as column ranges of one [rows, 2 D] matrix pass the overlap
    check (and then find no device); one column more does not."""
    ok = fwd(r=at(5), h=at(5, 2 * COLS), ld_r=2 * COLS, ld_h=2 * COLS)
    assert lib.zero1_block_norm_forward(cfg(), ok, None) == ECUDA
    bad = fwd(r=at(5), h=at(5, 2 * COLS - 2), ld_r=2 * COLS, ld_h=2 * COLS)
    assert lib.zero1_block_norm_forward(cfg(), bad, None) == EINVAL


@pytest.mark.parametrize("change,code", [
    (dict(dh=0), EINVAL), (dict(dx=0), EINVAL), (dict(dy=0), EINVAL), (dict(r=0), EINVAL), (dict(y=0), EINVAL),
    (dict(rstd_post=0), EINVAL), (dict(rstd_pre=0), EINVAL), (dict(w_post=0), EINVAL), (dict(w_pre=0), EINVAL),
    (dict(dgate=at(13)), EINVAL), (dict(dx=at(10, 1)), EALIGN), (dict(dw_pre=at(12, 2)), EALIGN),
    (dict(ld_dy=COLS - 1), EINVAL), (dict(dy=at(10)), EINVAL), (dict(dw_post=at(12)), EINVAL), (dict(dx=at(4)), EINVAL),
    (dict(dy=at(2)), EINVAL), (dict(dx=at(2, 400)), EINVAL), (dict(dw_pre=at(30)), EINVAL),
])
def test_backward_refusals(lib, change, code):
    assert lib.zero1_block_norm_backward(cfg(), bwd(**change), at(30), 1 << 22, None) == code, reason(lib)


def test_backward_saved_activation_refusals(lib):
    k, other = ckpt(), ckpt(cols=199)
    a, b = ctypes.addressof(k), ctypes.addressof(other)
    run = lambda **kw: lib.zero1_block_norm_backward(cfg(), bwd(**kw), at(30), 1 << 22, None)  # noqa: E731
    assert run(y8=a) == EINVAL                       # both y and y8
    assert run(r8=a) == EINVAL                       # both r and r8
    assert run(r=0, r8=b) == EINVAL and "100 x 199" in reason(lib)
    assert run(w_post=0, rstd_post=0, dw_post=0, w_pre=0, rstd_pre=0, dw_pre=0, dh=0, r=0, dr=0, y=0) == EINVAL
    assert "neither" in reason(lib)


# ----------------------------------------------------------- weight gradient --

def test_weight_grad_refusals(lib):
    k = ckpt()

    def run(dy=at(1), ld_dy=64, n=64, x8=None, col=0, ct=0, dw=at(2), ld_dw=200, out=BF16):
        return lib.zero1_weight_grad(dy, ld_dy, n, ctypes.addressof(k) if x8 is None else x8, col, ct, dw, ld_dw, out, 0,
                                     None, 0, None)
    assert run(n=0) == EINVAL
    assert run(dy=0) == EINVAL
    assert run(dw=0) == EINVAL
    assert run(out=2) == EINVAL
    assert run(col=at(3), ct=5) == EINVAL
    assert run(x8=0) == EINVAL
    assert run(dy=at(1, 1)) == EALIGN
    assert run(dw=at(2, 2), out=F32) == EALIGN
    assert run(col=at(3, 2), ct=F32) == EALIGN
    assert run(ld_dy=-64) == EINVAL
    assert run(ld_dw=199) == EINVAL
    assert run(dw=at(1)) == EINVAL                    # dw over dy
    assert run(dw=at(20)) == EINVAL                   # dw over the codes
    assert run(col=at(2, 8)) == EINVAL                # dw over col_scale
    out = ctypes.c_int64()
    assert lib.zero1_weight_grad_workspace(-1, 4, 4, at(1), 4, ctypes.addressof(out)) == EINVAL
    assert lib.zero1_weight_grad_workspace(4, 4, 4, at(1), 4, None) == EINVAL
    assert lib.zero1_weight_grad_workspace(1 << 32, 4, 4, at(1), 4, ctypes.addressof(out)) == ERANGE


# ------------------------------------------------------------------- binding --

def test_binding_refuses_host_tensors_and_wrong_types():
    t = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor or a pinned host tensor"):
        z.new_checkpoint(4, 8, "cpu")
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        z.zero1_checkpoint_pack(t.half(), None)
    with pytest.raises(ValueError, match="expected a matrix"):
        z.zero1_checkpoint_pack(t[0], None)
    with pytest.raises(TypeError, match="expected a Checkpoint8"):
        z.zero1_checkpoint_pack(t, None)
    with pytest.raises(ValueError, match="gate_act"):
        z.zero1_block_norm_workspace(z.BlockNorm(gate_act="tanh"), 4, 8)
