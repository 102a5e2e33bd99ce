"""The global gradient norm and clipping: over lists of tensors, and in the
sharded step (include/zero1.h has the formulas).

Argument marshalling only, as in _lib and block.  The norm stays on the device
as its square, a float64 tensor of one element.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import block as _block
from ._lib import AdamW, Plan, _AdamWStruct, _check_rc, _dev, _range, _replicas
from .block import _CODES, _call_with, _get_device, _launch_stream, _usable

_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float

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


_Tensor = torch.Tensor
_BF16, _F32, _F64 = torch.bfloat16, torch.float32, torch.float64


def _table(tensors, what: str) -> bytes:
    """zero1_tensor_t of each tensor, packed."""
    device = _get_device()
    rows = []
    for t in tensors:
        if isinstance(t, _Tensor) and t.get_device() == device and t.is_contiguous():
            dtype = t.dtype
            if dtype is _BF16:
                rows += (t.data_ptr(), t.numel(), 0)
                continue
            if dtype is _F32:
                rows += (t.data_ptr(), t.numel(), 1)
                continue
        rows += _unusual(t, f"{what}[{len(rows) // 3}]")
    return struct.pack("=" + "Qqq" * (len(rows) // 3), *rows)


def _unusual(t, what: str):
    """The same for what is pinned, or wrong."""
    _usable(t, what)
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{what}: expected bfloat16 or float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: must be contiguous")
    return t.data_ptr(), t.numel(), code


def _ptr(t, dtype, numel: int, what: str) -> int:
    """_dev, by the short way for a usual tensor; on the current device, or pinned."""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == _get_device() and t.is_contiguous()
            and t.numel() >= numel):
        return t.data_ptr()
    _usable(t, what)
    return _dev(t, dtype, numel, what)


def _scalar(t, dtype, numel: int, what: str):
    return None if t is None else _ptr(t, dtype, numel, what)


def _grads(plan: Plan, grads, nv: int):
    """The replicas' gradient pointers, as a host array."""
    _replicas(plan, grads, "grads")
    return struct.pack(f"={plan.M}Q", *[_ptr(t, _BF16, nv, "a replica's gradient") for t in grads])


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
    _check_rc(_call_with(workspace, nbytes, stream, lib.zero1_grad_sumsq, table, n, _ptr(sumsq, _F64, 1, "sumsq"),
                         _scalar(norms, _F32, n, "norms"), 1 if accumulate else 0))


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
    _check_rc(_lib().zero1_grad_clip(table, out, n, _ptr(sumsq, _F64, 1, "sumsq"), max_norm,
                                     _scalar(norm, _F32, 1, "norm"), _launch_stream(stream)))


def zero1_shard_grad_sumsq(plan: Plan, shard_begin: int, shard_end: int, grads, hp: AdamW, sumsq: torch.Tensor, *,
                           sums: torch.Tensor | None = None, accumulate: bool = False,
                           workspace: torch.Tensor | None = None, stream=None) -> None:
    """Sum of squares of the summed, unscaled gradients of shards [shard_begin,
    shard_end), written to sumsq (float64, one element) or added to it.  sums:
    fp32, L elements, keeps the replicas' sums for zero1_step_clipped."""
    _, L, nv = _range(plan, shard_begin, shard_end)
    nbytes = zero1_shard_grad_sumsq_workspace() if workspace is None else 0
    _check_rc(_call_with(workspace, nbytes, stream, _lib().zero1_shard_grad_sumsq, ctypes.byref(plan), shard_begin,
                         shard_end, _grads(plan, grads, nv), ctypes.byref(hp.c_struct()), _ptr(sumsq, _F64, 1, "sumsq"),
                         _scalar(sums, _F32, L, "sums"), 1 if accumulate else 0))


@functools.cache
def zero1_shard_grad_sumsq_workspace() -> int:
    """Bytes of scratch memory that zero1_shard_grad_sumsq needs, the same for every plan."""
    out = _i64()
    _check_rc(_lib().zero1_shard_grad_sumsq_workspace(ctypes.addressof(out)))
    return out.value


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
    g = _grads(plan, grads, nv) if sums is None else None
    names = ("master", "m", "v")
    state = [_ptr(t, _F32, L, k) for t, k in zip((master, m, v), names)]
    if out is None:
        to = state
    else:
        if len(out) != 3:
            raise ValueError("out: expected three tensors (master, m, v)")
        to = [_ptr(t, _F32, L, f"out {k}") for t, k in zip(out, names)]
    _check_rc(_lib().zero1_step_clipped(
        ctypes.byref(plan), shard_begin, shard_end, g, _scalar(sums, _F32, L, "sums"), *state, *to,
        _ptr(params, _BF16, nv, "params"), ctypes.byref(hp.c_struct()), _ptr(sumsq, _F64, 1, "sumsq"),
        max_norm, _scalar(norm, _F32, 1, "norm"), _scalar(overflow_flag, torch.int32, 1, "overflow_flag"),
        _launch_stream(stream)))
