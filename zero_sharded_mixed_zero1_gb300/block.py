"""Operators of a training block next to the optimizer step: block norms with
gate and residual scale, 8-bit activation checkpoints, and the weight gradient
taken from a checkpoint (include/zero1.h has the formulas).

Argument marshalling only, as in _lib.  Matrices are 2-D tensors whose columns
are contiguous; rows may be strided.  Every call launches on the current
stream unless `stream` is given.  Workspaces are allocated with the calling
stream's allocator when the caller passes none.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

import torch

from ._lib import ZERO1_DTYPE_BF16, ZERO1_DTYPE_F32, _check_rc, _stream, load

_CODES = {torch.bfloat16: ZERO1_DTYPE_BF16, torch.float32: ZERO1_DTYPE_F32}
_vp, _i64, _i32, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float

CHECKPOINT_BLOCK = 128
BLOCK_NORM_MAX_COLS = 16384
_GATE_NONE, _GATE_CHANNEL, _GATE_TOKEN, _GATE_FULL = 0, 1, 2, 3
_GATE_ACTS = {"linear": 0, "sigmoid": 1}


# The C structs of include/zero1.h, packed by hand (pointers as integers, 0 for
# NULL): a few times faster than filling ctypes structures, which shows on
# small calls.
_CKPT = struct.Struct("=QQqqqq")
_CFG = struct.Struct("=qqff8i")
_FWD = struct.Struct("=11Q5q")
_BWD = struct.Struct("=16Q8q")

_Tensor = torch.Tensor
_ready = None


def _lib():
    global _ready
    if _ready is None:
        lib = load()
        lib.zero1_checkpoint_pack.argtypes = [_vp, _i64, _i32, _vp, _vp]
        lib.zero1_checkpoint_unpack.argtypes = [_vp, _vp, _i64, _i32, _vp]
        lib.zero1_block_norm_forward.argtypes = [_vp, _vp, _vp]
        lib.zero1_block_norm_workspace.argtypes = [_vp, _vp]
        lib.zero1_block_norm_backward.argtypes = [_vp, _vp, _vp, _i64, _vp]
        lib.zero1_weight_grad_workspace.argtypes = [_i64, _i64, _i64, _vp, _i64, _vp]
        lib.zero1_weight_grad.argtypes = [_vp, _i64, _i64, _vp, _vp, _i32, _vp, _i64, _i32, _i32, _vp, _i64, _vp]
        _ready = lib
    return _ready


_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch_stream(stream) -> int:
    """_stream, by the short way for the current stream."""
    if stream is None and _raw_stream is not None:
        return _raw_stream(_get_device())
    return _stream(stream)


def _usable(t: torch.Tensor, what: str) -> None:
    """Raises unless the kernels can address t: on the current device, or pinned."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    device = t.get_device()  # -1 on the host
    if device >= 0:
        if device != _get_device():
            raise ValueError(f"{what}: on cuda:{device}, the current device is cuda:{_get_device()}")
    elif not (t.device.type == "cpu" and t.is_pinned()):
        raise ValueError(f"{what}: must be a CUDA tensor or a pinned host tensor")


def _matrix(t: torch.Tensor, shape: tuple, dtype, what: str) -> tuple[int, int]:
    """(pointer, row stride) of a tensor of this shape with contiguous columns."""
    if isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == _get_device():
        ld, step = t.stride()
        if step == 1:
            return t.data_ptr(), ld
    _usable(t, what)  # the long way, for what is unusual or wrong
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{what}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{what}: columns must be contiguous")
    return t.data_ptr(), ld


def _vector(t: torch.Tensor, numel: int, dtype, what: str) -> int:
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == (numel,) and t.stride() == (1,)
            and t.get_device() == _get_device()):
        return t.data_ptr()
    _usable(t, what)
    if t.dtype is not dtype:
        raise TypeError(f"{what}: expected {dtype}, got {t.dtype}")
    if t.shape != (numel,):
        raise ValueError(f"{what}: expected shape ({numel},), got {tuple(t.shape)}")
    if numel > 1 and t.stride(0) != 1:
        raise ValueError(f"{what}: must be contiguous")
    return t.data_ptr()


def _optional(t, numel: int, dtype, what: str) -> int:
    return 0 if t is None else _vector(t, numel, dtype, what)


def _code(t: torch.Tensor, what: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"{what}: expected bfloat16 or float32, got {t.dtype}")
    return c


def _dims(t: torch.Tensor, what: str) -> tuple[int, int]:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{what}: expected a matrix, got shape {tuple(t.shape)}")
    return t.shape


class Checkpoint8:
    """An 8-bit checkpoint of a [rows, cols] activation: `codes`, a uint8
    tensor [rows, >= cols rounded up to 128] of e4m3 codes, and `exps`, a uint8
    tensor [cols / 128 rounded up, >= rows rounded up to 128] of biased
    power-of-two scales.  Make one with new_checkpoint, or from tensors that
    the caller owns."""
    __slots__ = ("rows", "cols", "codes", "exps", "c")

    def __init__(self, rows: int, cols: int, codes: torch.Tensor, exps: torch.Tensor):
        for t, what in ((codes, "codes"), (exps, "exps")):
            _usable(t, what)
            if t.dtype is not torch.uint8:
                raise TypeError(f"{what}: expected torch.uint8, got {t.dtype}")
            if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
                raise ValueError(f"{what}: expected a matrix with contiguous columns")
        blocks = -(-cols // CHECKPOINT_BLOCK)
        (h, w), (eh, ew) = codes.shape, exps.shape
        if h < rows or w < blocks * CHECKPOINT_BLOCK:
            raise ValueError(f"codes: shape {(h, w)} is too small for {rows} x {cols}")
        if eh < blocks or ew < -(-rows // CHECKPOINT_BLOCK) * CHECKPOINT_BLOCK:
            raise ValueError(f"exps: shape {(eh, ew)} is too small for {rows} x {cols}")
        self.rows, self.cols, self.codes, self.exps = rows, cols, codes, exps
        self.c = ctypes.create_string_buffer(
            _CKPT.pack(codes.data_ptr(), exps.data_ptr(), codes.stride(0), exps.stride(0), rows, cols), _CKPT.size)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.exps.numel()


def new_checkpoint(rows: int, cols: int, device) -> Checkpoint8:
    """Storage for the checkpoint of a [rows, cols] activation."""
    blocks = -(-cols // CHECKPOINT_BLOCK)
    padded = -(-rows // CHECKPOINT_BLOCK) * CHECKPOINT_BLOCK
    return Checkpoint8(rows, cols, torch.empty((rows, blocks * CHECKPOINT_BLOCK), dtype=torch.uint8, device=device),
                       torch.empty((blocks, padded), dtype=torch.uint8, device=device))


def _ckpt(k, shape: tuple, what: str) -> int:
    if not isinstance(k, Checkpoint8):
        raise TypeError(f"{what}: expected a Checkpoint8")
    if (k.rows, k.cols) != shape:
        raise ValueError(f"{what}: checkpoint of {k.rows} x {k.cols}, expected {shape[0]} x {shape[1]}")
    return ctypes.addressof(k.c)


def zero1_checkpoint_pack(x: torch.Tensor, ckpt: Checkpoint8, stream=None) -> None:
    """Pack x (bf16 or fp32, [rows, cols]) into ckpt."""
    code, shape = _code(x, "x"), _dims(x, "x")
    k = _ckpt(ckpt, shape, "ckpt")
    p, ld = _matrix(x, shape, x.dtype, "x")
    _check_rc(_lib().zero1_checkpoint_pack(p, ld, code, k, _launch_stream(stream)))


def zero1_checkpoint_unpack(ckpt: Checkpoint8, out: torch.Tensor, stream=None) -> torch.Tensor:
    """Write the values ckpt stands for into out (bf16 or fp32, [rows, cols])."""
    code, shape = _code(out, "out"), _dims(out, "out")
    k = _ckpt(ckpt, shape, "ckpt")
    p, ld = _matrix(out, shape, out.dtype, "out")
    _check_rc(_lib().zero1_checkpoint_unpack(k, p, ld, code, _launch_stream(stream)))
    return out


@dataclass(frozen=True)
class BlockNorm:
    """eps, residual scale and gate activation ("linear" or "sigmoid") of a
    block's norms (zero1_block_norm_t)."""
    eps: float = 1e-6
    residual_scale: float = 1.0
    gate_act: str = "linear"


def _gate(gate, shape: tuple):
    """(kind, dtype code, pointer, ld) from the gate's shape: (cols,),
    (rows, 1) or (rows, cols); with one column the last two are the same, a
    gate per element."""
    if gate is None:
        return _GATE_NONE, 0, 0, 0
    code = _code(gate, "gate")
    if gate.dim() == 1:
        return _GATE_CHANNEL, code, _vector(gate, shape[1], gate.dtype, "gate"), 0
    if gate.shape == (shape[0], 1) and shape[1] != 1:
        return (_GATE_TOKEN, code, *_matrix(gate, (shape[0], 1), gate.dtype, "gate"))
    return (_GATE_FULL, code, *_matrix(gate, shape, gate.dtype, "gate"))


def _params(w_post, w_pre, cols: int):
    """(dtype code, pointers) of the two weights, which share a type."""
    w = w_post if w_post is not None else w_pre
    if w is None:
        return ZERO1_DTYPE_BF16, 0, 0
    code, dtype = _code(w, "w_post" if w is w_post else "w_pre"), w.dtype
    return code, _optional(w_post, cols, dtype, "w_post"), _optional(w_pre, cols, dtype, "w_pre")


def _cfg(cfg: BlockNorm, shape, act, res, param, gate, grad, kind, accumulate) -> bytes:
    a = _GATE_ACTS.get(cfg.gate_act)
    if a is None:
        raise ValueError(f"gate_act: {cfg.gate_act!r} is neither 'linear' nor 'sigmoid'")
    return _CFG.pack(*shape, cfg.eps, cfg.residual_scale, act, res, param, gate, grad, kind, a, accumulate)


def zero1_block_norm_forward(cfg: BlockNorm, y, x, r, h=None, rstd_post=None, rstd_pre=None, *, w_post=None, w_pre=None,
                             gate=None, y8: Checkpoint8 | None = None, r8: Checkpoint8 | None = None,
                             stream=None) -> None:
    """r = x + residual_scale * gate * norm_post(y); h = norm_pre(r).

    y, h: [T, D] of one type; x, r: [T, D] of one type (r may be x).  w_post or
    w_pre None leaves that norm out, with its rstd (and h).  gate: None, or of
    shape (D,), (T, 1) or (T, D).  rstd_post, rstd_pre: fp32 [T], written.
    y8, r8: checkpoints of the normalised rows, written when given."""
    shape = _dims(y, "y")
    rows, cols = shape
    act, res, ta, tr = _code(y, "y"), _code(x, "x"), y.dtype, x.dtype
    py, ly = _matrix(y, shape, ta, "y")
    px, lx = _matrix(x, shape, tr, "x")
    pr, lr = _matrix(r, shape, tr, "r")
    ph, lh = (0, 0) if h is None else _matrix(h, shape, ta, "h")
    kind, gcode, pg, lg = _gate(gate, shape)
    pcode, wq, wp = _params(w_post, w_pre, cols)
    c = _cfg(cfg, shape, act, res, pcode, gcode, 0, kind, 0)
    io = _FWD.pack(py, px, wq, wp, pg, pr, ph, _optional(rstd_post, rows, torch.float32, "rstd_post"),
                   _optional(rstd_pre, rows, torch.float32, "rstd_pre"), 0 if y8 is None else _ckpt(y8, shape, "y8"),
                   0 if r8 is None else _ckpt(r8, shape, "r8"), ly, lx, lg, lr, lh)
    _check_rc(_lib().zero1_block_norm_forward(c, io, _launch_stream(stream)))


def _scratch(nbytes: int, stream) -> torch.Tensor:
    """Scratch memory on the current device, of the stream that will use it."""
    device = torch.device("cuda", _get_device())
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    st = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(st):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _workspace(workspace, nbytes: int, stream):
    """(pointer, bytes, tensor) of the caller's workspace or a new one; the
    tensor is kept until the call has been made, and its memory then goes back
    to the stream that uses it.  Always device memory, wherever the call's
    tensors are: host memory would be freed while the kernels still write it."""
    if workspace is None:
        if not nbytes:
            return None, 0, None
        workspace = _scratch(nbytes, stream)
        return workspace.data_ptr(), nbytes, workspace
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace: expected a torch.Tensor")
    if workspace.dtype is not torch.uint8 or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous CUDA uint8 tensor")
    if workspace.get_device() != _get_device():
        raise ValueError(f"workspace: on {workspace.device}, the current device is cuda:{_get_device()}")
    return workspace.data_ptr(), workspace.numel(), workspace


_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _call_with(workspace, nbytes: int, stream, fn, *args) -> int:
    """fn(*args, workspace, its bytes, stream): with the caller's workspace, or
    with memory of the calling stream that goes back to it after the call, from
    the allocator itself where that is there (a few microseconds less than a
    tensor)."""
    st = _launch_stream(stream)
    if workspace is not None or not nbytes or _raw_alloc is None or _raw_delete is None:
        ws, nbytes, keep = _workspace(workspace, nbytes, stream)
        return fn(*args, ws, nbytes, st)
    ws = _raw_alloc(nbytes, st)
    try:
        return fn(*args, ws, nbytes, st)
    finally:
        _raw_delete(ws)


def zero1_block_norm_workspace(cfg: BlockNorm, rows: int, cols: int) -> int:
    """Bytes of scratch memory that zero1_block_norm_backward needs."""
    c = _cfg(cfg, (rows, cols), 0, 0, 0, 0, 0, 0, 0)
    n = _i64()
    _check_rc(_lib().zero1_block_norm_workspace(c, ctypes.addressof(n)))
    return n.value


def zero1_block_norm_backward(cfg: BlockNorm, dh, dr, y, r, rstd_post, rstd_pre, dy, dx, *, w_post=None, w_pre=None,
                              gate=None, dw_post=None, dw_pre=None, dgate=None, accumulate: bool = False,
                              workspace: torch.Tensor | None = None, stream=None) -> None:
    """Gradients of zero1_block_norm_forward from dh and dr (dr None: zero).

    y, r: the saved activations, each either the tensor of the forward call or
    its checkpoint (Checkpoint8) of the normalised rows.  Writes dy and dx (dy
    may be dh, dx may be dr), dw_post and dw_pre [D] and dgate (the gate's
    shape; a [T, D] dgate has the gate's type, the other sums share one type),
    each only if given.  accumulate adds to dw_post, dw_pre and a (D,) dgate."""
    shape = _dims(dy, "dy")
    rows, cols = shape
    act, res, ta, tr = _code(dy, "dy"), _code(dx, "dx"), dy.dtype, dx.dtype
    pdy, ldy = _matrix(dy, shape, ta, "dy")
    pdx, ldx = _matrix(dx, shape, tr, "dx")
    pdh, ldh = (0, 0) if dh is None else _matrix(dh, shape, ta, "dh")
    pdr, ldr = (0, 0) if dr is None else _matrix(dr, shape, tr, "dr")
    py = pr = py8 = pr8 = ly = lr = 0
    if isinstance(y, Checkpoint8):
        py8 = _ckpt(y, shape, "y")
    elif y is not None:
        py, ly = _matrix(y, shape, ta, "y")
    if isinstance(r, Checkpoint8):
        pr8 = _ckpt(r, shape, "r")
    elif r is not None:
        pr, lr = _matrix(r, shape, tr, "r")
    kind, gcode, pg, lg = _gate(gate, shape)
    pcode, wq, wp = _params(w_post, w_pre, cols)
    first = dw_post if dw_post is not None else dw_pre if dw_pre is not None else dgate if kind != _GATE_FULL else None
    wcode, tw = (0, None) if first is None else (_code(first, "a weight gradient"), first.dtype)
    pgd = lgd = 0
    if dgate is not None:
        if gate is None:
            raise ValueError("dgate: there is no gate")
        if kind == _GATE_CHANNEL:
            pgd = _vector(dgate, cols, tw, "dgate")
        else:
            pgd, lgd = _matrix(dgate, gate.shape, gate.dtype if kind == _GATE_FULL else tw, "dgate")
    c = _cfg(cfg, shape, act, res, pcode, gcode, wcode, kind, 1 if accumulate else 0)
    io = _BWD.pack(pdh, pdr, py, pr, wq, wp, pg, _optional(rstd_post, rows, torch.float32, "rstd_post"),
                   _optional(rstd_pre, rows, torch.float32, "rstd_pre"), py8, pr8, pdy, pdx,
                   _optional(dw_post, cols, tw, "dw_post"), _optional(dw_pre, cols, tw, "dw_pre"), pgd,
                   ldh, ldr, ly, lr, lg, ldy, ldx, lgd)
    lib = _lib()
    nbytes = 0
    if first is not None and workspace is None:
        need = _i64()
        _check_rc(lib.zero1_block_norm_workspace(c, ctypes.addressof(need)))
        nbytes = need.value
    ws, nbytes, keep = _workspace(workspace, nbytes, stream)
    _check_rc(lib.zero1_block_norm_backward(c, io, ws, nbytes, _launch_stream(stream)))


def zero1_weight_grad_workspace(dy: torch.Tensor, cols: int) -> int:
    """Bytes of scratch memory that zero1_weight_grad needs for this dy and an
    input of `cols` columns."""
    shape = _dims(dy, "dy")
    p, ld = _matrix(dy, shape, torch.bfloat16, "dy")
    out = _i64()
    _check_rc(_lib().zero1_weight_grad_workspace(*shape, cols, p, ld, ctypes.addressof(out)))
    return out.value


def zero1_weight_grad(dy, x8: Checkpoint8, dw, *, col_scale=None, accumulate: bool = False,
                      workspace: torch.Tensor | None = None, stream=None) -> None:
    """dw (+)= dy^T X * col_scale, X the values of x8: dy bf16 [T, N], x8 a
    checkpoint of [T, K], dw [N, K] bf16 or fp32 (for instance a view into a
    replica's flat gradient buffer), col_scale [K] bf16 or fp32."""
    shape = _dims(dy, "dy")
    rows, n = shape
    pdy, ld = _matrix(dy, shape, torch.bfloat16, "dy")
    k = _ckpt(x8, (rows, x8.cols if isinstance(x8, Checkpoint8) else 0), "x8")
    cols = x8.cols
    code = _code(dw, "dw")
    pw, lw = _matrix(dw, (n, cols), dw.dtype, "dw")
    pc, ccode = 0, 0
    if col_scale is not None:
        ccode = _code(col_scale, "col_scale")
        pc = _vector(col_scale, cols, col_scale.dtype, "col_scale")
    lib = _lib()
    nbytes = 0
    if workspace is None:
        need = _i64()
        _check_rc(lib.zero1_weight_grad_workspace(rows, n, cols, pdy, ld, ctypes.addressof(need)))
        nbytes = need.value
    ws, nbytes, keep = _workspace(workspace, nbytes, stream)
    _check_rc(lib.zero1_weight_grad(pdy, ld, n, k, pc, ccode, pw, lw, code, 1 if accumulate else 0, ws, nbytes,
                                    _launch_stream(stream)))
