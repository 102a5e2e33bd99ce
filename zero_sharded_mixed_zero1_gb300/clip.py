"""The global gradient norm and clipping: over lists of tensors, and in the
sharded step (include/zero1.h has the formulas).

Argument marshalling only, as in _lib and block.  The norm stays on the device
as its square, a float64 tensor of one element.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import block as _block
from ._lib import AdamW, Plan, _AdamWStruct, _check_rc, _dev, _ptrs, _range, _replicas
from .block import _CODES, _get_device, _launch_stream, _usable, _workspace

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
SHARD_WORKSPACE = 8 * 2048

_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = _block._lib()
        P, A = ctypes.POINTER(Plan), ctypes.POINTER(_AdamWStruct)
        lib.zero1_grad_sumsq_workspace.argtypes = [_vp, _i32, _vp]
        lib.zero1_grad_sumsq.argtypes = [_vp, _i32, _vp, _vp, _i32, _vp, _i64, _vp]
        lib.zero1_grad_clip.argtypes = [_vp, _vp, _i32, _vp, _f32, _vp, _vp]
        lib.zero1_shard_grad_sumsq_workspace.argtypes = [_vp]
        lib.zero1_shard_grad_sumsq.argtypes = [P, _i32, _i32, _vp, A, _vp, _vp, _i32, _vp, _i64, _vp]
        lib.zero1_step_clipped.argtypes = [P, _i32, _i32, *[_vp] * 9, A, _vp, _f32, _vp, _vp, _vp]
        _ready = lib
    return _ready


def _table(tensors, what: str) -> bytes:
    """zero1_tensor_t of each tensor, packed."""
    device, rows = _get_device(), []
    for i, t in enumerate(tensors):
        code = _CODES.get(t.dtype) if isinstance(t, torch.Tensor) else None
        if code is None or t.get_device() != device or not t.is_contiguous():
            _usable(t, f"{what}[{i}]")  # the long way, for what is unusual or wrong
            if code is None:
                raise TypeError(f"{what}[{i}]: expected bfloat16 or float32, got {t.dtype}")
            if not t.is_contiguous():
                raise ValueError(f"{what}[{i}]: must be contiguous")
        rows += (t.data_ptr(), t.numel(), code)
    return struct.pack("=" + "Qqq" * (len(rows) // 3), *rows)


def _scalar(t, dtype, numel: int, what: str):
    return None if t is None else _dev(t, dtype, numel, what)


def zero1_grad_sumsq(tensors, sumsq: torch.Tensor, *, norms: torch.Tensor | None = None, accumulate: bool = False,
                     workspace: torch.Tensor | None = None, stream=None) -> None:
    """Sum of squares over a list of gradients (contiguous bf16 or fp32 tensors
    of any shape), written to sumsq (float64, one element), or added to it with
    accumulate.  norms: fp32, one element per tensor, gets each tensor's norm."""
    tensors = list(tensors)
    table, n, lib = _table(tensors, "tensors"), len(tensors), _lib()
    nbytes = 0
    if workspace is None:
        need = _i64()
        _check_rc(lib.zero1_grad_sumsq_workspace(table, n, ctypes.addressof(need)))
        nbytes = need.value
    ws, nbytes, keep = _workspace(workspace, nbytes, stream)
    _check_rc(lib.zero1_grad_sumsq(table, n, _dev(sumsq, torch.float64, 1, "sumsq"),
                                   _scalar(norms, torch.float32, n, "norms"), 1 if accumulate else 0, ws, nbytes,
                                   _launch_stream(stream)))


def zero1_grad_sumsq_workspace(tensors) -> int:
    """Bytes of scratch memory that zero1_grad_sumsq needs for this list."""
    tensors, out = list(tensors), _i64()
    _check_rc(_lib().zero1_grad_sumsq_workspace(_table(tensors, "tensors"), len(tensors), ctypes.addressof(out)))
    return out.value


def zero1_grad_clip(tensors, sumsq: torch.Tensor, max_norm: float, *, outs=None, norm: torch.Tensor | None = None,
                    stream=None) -> None:
    """Every gradient times min(1, max_norm / (sqrt(sumsq) + 1e-6)), in place or
    into `outs` (tensors of the same sizes and types).  norm: fp32, one element,
    gets the norm.  Gradients whose sum of squares is not finite stay as they are."""
    tensors = list(tensors)
    n, table, out = len(tensors), _table(tensors, "tensors"), None
    if outs is not None:
        outs = list(outs)
        if len(outs) != n:
            raise ValueError(f"outs: expected {n} tensors, got {len(outs)}")
        out = _table(outs, "outs")
    _check_rc(_lib().zero1_grad_clip(table, out, n, _dev(sumsq, torch.float64, 1, "sumsq"), max_norm,
                                     _scalar(norm, torch.float32, 1, "norm"), _launch_stream(stream)))


def zero1_shard_grad_sumsq(plan: Plan, shard_begin: int, shard_end: int, grads, hp: AdamW, sumsq: torch.Tensor, *,
                           sums: torch.Tensor | None = None, accumulate: bool = False,
                           workspace: torch.Tensor | None = None, stream=None) -> None:
    """Sum of squares of the summed, unscaled gradients of shards [shard_begin,
    shard_end), written to sumsq (float64, one element) or added to it.  sums:
    fp32, L elements, keeps the replicas' sums for zero1_step_clipped."""
    _replicas(plan, grads, "grads")
    _, L, nv = _range(plan, shard_begin, shard_end)
    ws, nbytes, keep = _workspace(workspace, SHARD_WORKSPACE, stream)
    _check_rc(_lib().zero1_shard_grad_sumsq(
        ctypes.byref(plan), shard_begin, shard_end, _ptrs(grads, torch.bfloat16, nv, "grads"), ctypes.byref(hp.c_struct()),
        _dev(sumsq, torch.float64, 1, "sumsq"), _scalar(sums, torch.float32, L, "sums"), 1 if accumulate else 0, ws, nbytes,
        _launch_stream(stream)))


def zero1_step_clipped(plan: Plan, shard_begin: int, shard_end: int, grads, master, m, v, params, hp: AdamW,
                       sumsq: torch.Tensor, max_norm: float, *, sums: torch.Tensor | None = None, out=None,
                       norm: torch.Tensor | None = None, overflow_flag: torch.Tensor | None = None, stream=None) -> None:
    """The fused step over shards [shard_begin, shard_end) with gradients
    clipped to a global norm of max_norm, of which sumsq (float64, one element)
    holds the square, summed over all shards and ranks.  sums: what
    zero1_shard_grad_sumsq kept (grads is then not read).  out: where the updated
    (master, m, v) go, by default in place.  norm: fp32, one element, gets the
    norm.  If sumsq is not finite, nothing else is written and overflow_flag set."""
    _, L, nv = _range(plan, shard_begin, shard_end)
    g = None
    if sums is None:
        _replicas(plan, grads, "grads")
        g = _ptrs(grads, torch.bfloat16, nv, "grads")
    names = ("master", "m", "v")
    state = [_dev(t, torch.float32, L, k) for t, k in zip((master, m, v), names)]
    if out is None:
        to = state
    else:
        if len(out) != 3:
            raise ValueError("out: expected three tensors (master, m, v)")
        to = [_dev(t, torch.float32, L, f"out {k}") for t, k in zip(out, names)]
    _check_rc(_lib().zero1_step_clipped(
        ctypes.byref(plan), shard_begin, shard_end, g, _scalar(sums, torch.float32, L, "sums"), *state, *to,
        _dev(params, torch.bfloat16, nv, "params"), ctypes.byref(hp.c_struct()), _dev(sumsq, torch.float64, 1, "sumsq"),
        max_norm, _scalar(norm, torch.float32, 1, "norm"), _scalar(overflow_flag, torch.int32, 1, "overflow_flag"),
        _launch_stream(stream)))
