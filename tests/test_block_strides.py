"""Row strides of the training-block calls that do not fit 64 bits of bytes,
without a GPU: they are refused, not taken for what they wrap round to."""
import ctypes

import pytest

from zero_sharded_mixed_zero1_gb300 import block as zb
from zero_sharded_mixed_zero1_gb300 import build as zbuild
from test_block_abi import BF16, COLS, EINVAL, ERANGE, F32, at, bwd, cfg, ckpt, fwd, reason

# times 2 or 4 bytes: 2^64 or 2^65 (wraps round to 0), 2^63 (to the most negative), 2^64 + 512 (to 512)
HUGE = [1 << 62, (1 << 63) - 1, 1 << 61, (1 << 62) + 256]


@pytest.fixture(scope="module")
def lib():
    zbuild.build()
    return zb._lib()


@pytest.mark.parametrize("ld", HUGE)
@pytest.mark.parametrize("types", [dict(), dict(act=F32, res=F32)])
def test_block_norms(lib, ld, types):
    for name in ("ld_y", "ld_x", "ld_r", "ld_h"):
        assert lib.zero1_block_norm_forward(cfg(**types), fwd(**{name: ld}), None) == ERANGE, (name, reason(lib))
        assert lib.zero1_block_norm_forward(cfg(**types), fwd(**{name: -ld}), None) == EINVAL, (name, reason(lib))
    for name in ("ld_dh", "ld_dr", "ld_y", "ld_r", "ld_dy", "ld_dx"):
        for sign, code in ((1, ERANGE), (-1, EINVAL)):
            call = lib.zero1_block_norm_backward(cfg(**types), bwd(**{name: sign * ld}), at(30), 1 << 22, None)
            assert call == code, (name, reason(lib))


@pytest.mark.parametrize("ld", HUGE)
@pytest.mark.parametrize("kind", [2, 3])
@pytest.mark.parametrize("gate_type", [BF16, F32])
def test_gates(lib, ld, kind, gate_type):
    c = cfg(kind=kind, gate=gate_type)
    good = dict(gate=at(13), ld_gate=COLS)
    assert lib.zero1_block_norm_forward(c, fwd(gate=at(13), ld_gate=ld), None) == ERANGE, reason(lib)
    assert lib.zero1_block_norm_backward(c, bwd(gate=at(13), ld_gate=ld), at(30), 1 << 22, None) == ERANGE, reason(lib)
    both = dict(good, dgate=at(14), ld_dgate=ld)
    assert lib.zero1_block_norm_backward(c, bwd(**both), at(30), 1 << 22, None) == ERANGE, reason(lib)


@pytest.mark.parametrize("ld", HUGE)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_checkpoints_and_weight_gradients(lib, ld, dtype):
    k = ckpt()
    a = ctypes.addressof(k)
    assert lib.zero1_checkpoint_pack(at(1), ld, dtype, a, None) == ERANGE, reason(lib)
    assert lib.zero1_checkpoint_unpack(a, at(1), ld, dtype, None) == ERANGE, reason(lib)
    grad = lambda ld_dy, n, ld_dw: lib.zero1_weight_grad(at(1), ld_dy, n, a, 0, 0, at(2), ld_dw, dtype, 0,  # noqa: E731
                                                         None, 0, None)
    assert grad(ld, 64, 200) == ERANGE, reason(lib)
    assert grad(64, 64, ld) == ERANGE, reason(lib)
    assert grad(64, ld, 200) == ERANGE, reason(lib)
