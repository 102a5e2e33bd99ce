"""The gated feed-forward block: forward, backward and input gradient, and
weight gradients from bf16 activations (include/zero1.h has the formulas).

Argument marshalling only, as in block: matrices are 2-D bf16 tensors whose
columns are contiguous; rows may be strided.  Every call launches on the
current stream unless `stream` is given; workspaces are allocated with the
calling stream's allocator when the caller passes none.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import block as _block
from ._lib import _check_rc
from .block import _call_with, _code, _dims, _matrix

_vp, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
_ACTS = {"silu": 0, "gelu": 1}
_FORWARD, _BACKWARD, _INPUT_GRAD = 0, 1, 2
_FFN = struct.Struct("=3q8Q8qi4x")  # zero1_gated_ffn_t

_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = _block._lib()
        lib.zero1_gated_ffn_workspace.argtypes = [_vp, _i32, _vp]
        for name in ("forward", "backward", "input_grad"):
            getattr(lib, "zero1_gated_ffn_" + name).argtypes = [_vp, _vp, _i64, _vp]
        lib.zero1_weight_grad_bf16_workspace.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _i32, _vp]
        lib.zero1_weight_grad_bf16.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp, _i64, _i32, _i32, _vp, _i64, _vp]
        _ready = lib
    return _ready


_NONE = (0, 0)


def _bf16(t, shape, what):
    return _matrix(t, shape, torch.bfloat16, what)


def _call(fn, kind: int, act: str, rows: int, d: int, f: int, h, w_gate, w_up, da, a, dg, du, dh, workspace, stream) -> None:
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act: {act!r} is neither 'silu' nor 'gelu'")
    m = (h, w_gate, w_up, da, a, dg, du, dh)
    c = _FFN.pack(rows, d, f, *[p for p, _ in m], *[ld for _, ld in m], code)
    lib = _lib()
    nbytes = 0
    if workspace is None:
        need = _i64()
        _check_rc(lib.zero1_gated_ffn_workspace(c, kind, ctypes.addressof(need)))
        nbytes = need.value
    _check_rc(_call_with(workspace, nbytes, stream, fn, c))


def _shapes(x, w_gate, what: str) -> tuple[int, int, int]:
    """(rows, d_model, d_ff) from a [rows, ...] matrix and w_gate."""
    rows = _dims(x, what)[0]
    f, d = _dims(w_gate, "w_gate")
    return rows, d, f


def zero1_gated_ffn_forward(h, w_gate, w_up, a, *, act: str = "silu", workspace: torch.Tensor | None = None,
                            stream=None) -> None:
    """a = act(h w_gate^T) * (h w_up^T): h bf16 [T, D], w_gate and w_up bf16
    [F, D], a bf16 [T, F], written.  act: "silu" or "gelu" (its tanh form)."""
    rows, d, f = _shapes(h, w_gate, "h")
    _call(_lib().zero1_gated_ffn_forward, _FORWARD, act, rows, d, f, _bf16(h, (rows, d), "h"),
          _bf16(w_gate, (f, d), "w_gate"), _bf16(w_up, (f, d), "w_up"), _NONE, _bf16(a, (rows, f), "a"), _NONE, _NONE, _NONE,
          workspace, stream)


def zero1_gated_ffn_backward(da, h, w_gate, w_up, dg, du, *, a=None, act: str = "silu",
                             workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of the two projections from that of a, [T, F] bf16 each:
    dg = da * u * act'(g) and du = da * act(g), with g = h w_gate^T and
    u = h w_up^T computed again.  dg may be da.  a, if given, is written as in
    the forward call."""
    rows, d, f = _shapes(h, w_gate, "h")
    _call(_lib().zero1_gated_ffn_backward, _BACKWARD, act, rows, d, f, _bf16(h, (rows, d), "h"),
          _bf16(w_gate, (f, d), "w_gate"), _bf16(w_up, (f, d), "w_up"), _bf16(da, (rows, f), "da"),
          _NONE if a is None else _bf16(a, (rows, f), "a"), _bf16(dg, (rows, f), "dg"), _bf16(du, (rows, f), "du"), _NONE,
          workspace, stream)


def zero1_gated_ffn_input_grad(dg, du, w_gate, w_up, dh, *, workspace: torch.Tensor | None = None, stream=None) -> None:
    """dh = dg w_gate + du w_up, [T, D] bf16, written; dg, du bf16 [T, F]."""
    rows, d, f = _shapes(dg, w_gate, "dg")
    _call(_lib().zero1_gated_ffn_input_grad, _INPUT_GRAD, "silu", rows, d, f, _NONE, _bf16(w_gate, (f, d), "w_gate"),
          _bf16(w_up, (f, d), "w_up"), _NONE, _NONE, _bf16(dg, (rows, f), "dg"), _bf16(du, (rows, f), "du"),
          _bf16(dh, (rows, d), "dh"), workspace, stream)


def zero1_gated_ffn_workspace(call: str, rows: int, w_gate, w_up, h=None, dg=None, du=None) -> int:
    """Bytes of scratch memory that a call ("forward", "backward" or
    "input_grad") needs for these weights and its other inputs of `rows` rows
    (h, or dg and du)."""
    kind = {"forward": _FORWARD, "backward": _BACKWARD, "input_grad": _INPUT_GRAD}.get(call)
    if kind is None:
        raise ValueError(f"call: {call!r} is none of 'forward', 'backward' and 'input_grad'")
    f, d = _dims(w_gate, "w_gate")
    g, u = _bf16(w_gate, (f, d), "w_gate"), _bf16(w_up, (f, d), "w_up")
    m = [_NONE, g, u, _NONE, _NONE, _NONE, _NONE, _NONE]
    if kind == _INPUT_GRAD:
        m[5], m[6] = _bf16(dg, (rows, f), "dg"), _bf16(du, (rows, f), "du")
    else:
        m[0] = _bf16(h, (rows, d), "h")
    out = _i64()
    _check_rc(_lib().zero1_gated_ffn_workspace(_FFN.pack(rows, d, f, *[p for p, _ in m], *[ld for _, ld in m], 0), kind,
                                               ctypes.addressof(out)))
    return out.value


def _grad_shapes(dy, x):
    rows, n = _dims(dy, "dy")
    k = _dims(x, "x")[1]
    return rows, n, k, *_bf16(dy, (rows, n), "dy"), *_bf16(x, (rows, k), "x")


def zero1_weight_grad_bf16_workspace(dy, x, dtype: torch.dtype) -> int:
    """Bytes of scratch memory that zero1_weight_grad_bf16 needs for these
    inputs and a gradient of this type."""
    rows, n, k, pdy, ldy, px, lx = _grad_shapes(dy, x)
    out = _i64()
    code = _code(torch.empty(0, dtype=dtype), "dtype")
    _check_rc(_lib().zero1_weight_grad_bf16_workspace(rows, n, k, pdy, ldy, px, lx, code, ctypes.addressof(out)))
    return out.value


def zero1_weight_grad_bf16(dy, x, dw, *, accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None) -> None:
    """dw (+)= dy^T x: dy bf16 [T, N], x bf16 [T, K], dw [N, K] bf16 or fp32
    (for instance a view into a replica's flat gradient buffer)."""
    rows, n, k, pdy, ldy, px, lx = _grad_shapes(dy, x)
    code = _code(dw, "dw")
    pw, lw = _matrix(dw, (n, k), dw.dtype, "dw")
    lib = _lib()
    nbytes = 0
    if workspace is None:
        need = _i64()
        _check_rc(lib.zero1_weight_grad_bf16_workspace(rows, n, k, pdy, ldy, px, lx, code, ctypes.addressof(need)))
        nbytes = need.value
    _check_rc(_call_with(workspace, nbytes, stream, lib.zero1_weight_grad_bf16, pdy, ldy, n, px, lx, k, rows, pw, lw, code,
                         1 if accumulate else 0))
