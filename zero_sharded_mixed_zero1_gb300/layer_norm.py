"""Layer norm with its residual, forward and backward (include/zero1.h has the
formulas).

Argument marshalling only, as in block: matrices are 2-D tensors whose columns
are contiguous; rows may be strided.  Every call launches on the current stream
unless `stream` is given; the workspace is allocated with the calling stream's
allocator when the caller passes none.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

import torch

from . import block as _block
from ._lib import ZERO1_DTYPE_BF16, _check_rc
from .block import Checkpoint8, _call_with, _ckpt, _code, _dims, _launch_stream, _matrix, _optional, _vector

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64
_CFG = struct.Struct("=qqff5i4x")  # zero1_layer_norm_t
_FWD = struct.Struct("=9Q4q")      # zero1_layer_norm_forward_t
_BWD = struct.Struct("=11Q5q")     # zero1_layer_norm_backward_t

_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = _block._lib()
        lib.zero1_layer_norm_forward.argtypes = [_vp, _vp, _vp]
        lib.zero1_layer_norm_workspace.argtypes = [_vp, _vp]
        lib.zero1_layer_norm_backward.argtypes = [_vp, _vp, _vp, _i64, _vp]
        _ready = lib
    return _ready


@dataclass(frozen=True)
class LayerNorm:
    """eps and residual scale of a layer norm (zero1_layer_norm_t)."""
    eps: float = 1e-5
    residual_scale: float = 1.0


def _pair(p, q, cols: int, what: str):
    """(dtype code, pointers) of two vectors of one type, each optional."""
    one = p if p is not None else q
    if one is None:
        return ZERO1_DTYPE_BF16, 0, 0
    a, b = what.split()
    code = _code(one, a if one is p else b)
    return code, _optional(p, cols, one.dtype, a), _optional(q, cols, one.dtype, b)


def zero1_layer_norm_forward(cfg: LayerNorm, x, h, mean, rstd, *, w=None, b=None, y=None, r=None,
                             r8: Checkpoint8 | None = None, stream=None) -> None:
    """r = x + residual_scale * y; h = w * (r - mean) * rstd + b.

    x, r: [T, D] of one type (r may be x); y, h: [T, D] of one type; without y
    the norm is of x itself, and there is no r.  w, b [D] of one type, each
    optional.  mean, rstd: fp32 [T], written.  r8: the checkpoint of the
    normalised rows, written when given."""
    shape = _dims(x, "x")
    rows, cols = shape
    act, res, ta, tr = _code(h, "h"), _code(x, "x"), h.dtype, x.dtype
    px, lx = _matrix(x, shape, tr, "x")
    ph, lh = _matrix(h, shape, ta, "h")
    py, ly = (0, 0) if y is None else _matrix(y, shape, ta, "y")
    pr, lr = (0, 0) if r is None else _matrix(r, shape, tr, "r")
    if (y is None) != (r is None):
        raise ValueError("y and r: both or neither")
    code, pw, pb = _pair(w, b, cols, "w b")
    c = _CFG.pack(rows, cols, cfg.eps, cfg.residual_scale, act, res, code, 0, 0)
    io = _FWD.pack(px, py, pw, pb, pr, ph, _vector(mean, rows, torch.float32, "mean"), _vector(rstd, rows, torch.float32, "rstd"),
                   0 if r8 is None else _ckpt(r8, shape, "r8"), lx, ly, lr, lh)
    _check_rc(_lib().zero1_layer_norm_forward(c, io, _launch_stream(stream)))


def zero1_layer_norm_workspace(rows: int, cols: int) -> int:
    """Bytes of scratch memory that zero1_layer_norm_backward needs."""
    n = _i64()
    _check_rc(_lib().zero1_layer_norm_workspace(_CFG.pack(rows, cols, 1.0, 1.0, 0, 0, 0, 0, 0), ctypes.addressof(n)))
    return n.value


def zero1_layer_norm_backward(cfg: LayerNorm, dh, dr, r, mean, rstd, dx, *, dy=None, w=None, dw=None, db=None,
                              accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of zero1_layer_norm_forward from dh and dr (dr None: zero).

    r: the saved rows, either the tensor (the forward call's r, or its x where it
    had no y) or the checkpoint (Checkpoint8) of the normalised rows.  Writes dx
    (may be dr) and, each only if given, dy = residual_scale * dx (may be dh), dw
    and db [D] of one type; accumulate adds to dw and db."""
    shape = _dims(dx, "dx")
    rows, cols = shape
    act, res, ta, tr = _code(dh, "dh"), _code(dx, "dx"), dh.dtype, dx.dtype
    pdx, ldx = _matrix(dx, shape, tr, "dx")
    pdh, ldh = _matrix(dh, shape, ta, "dh")
    pdr, ldr = (0, 0) if dr is None else _matrix(dr, shape, tr, "dr")
    pdy, ldy = (0, 0) if dy is None else _matrix(dy, shape, ta, "dy")
    pr = pr8 = lr = 0
    if isinstance(r, Checkpoint8):
        pr8 = _ckpt(r, shape, "r")
    else:
        pr, lr = _matrix(r, shape, tr, "r")
    pcode, pw = (ZERO1_DTYPE_BF16, 0) if w is None else (_code(w, "w"), _vector(w, cols, w.dtype, "w"))
    gcode, pdw, pdb = _pair(dw, db, cols, "dw db")
    c = _CFG.pack(rows, cols, cfg.eps, cfg.residual_scale, act, res, pcode, gcode, 1 if accumulate else 0)
    io = _BWD.pack(pdh, pdr, pr, pw, _vector(mean, rows, torch.float32, "mean"), _vector(rstd, rows, torch.float32, "rstd"), pr8,
                   pdx, pdy, pdw, pdb, ldh, ldr, lr, ldx, ldy)
    lib = _lib()
    nbytes = 0
    if workspace is None and (pdw or pdb):
        need = _i64()
        _check_rc(lib.zero1_layer_norm_workspace(c, ctypes.addressof(need)))
        nbytes = need.value
    _check_rc(_call_with(workspace, nbytes, stream, lib.zero1_layer_norm_backward, c, io))
