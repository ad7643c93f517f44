"""The operators of a residual block around a layer and of its training step (C ABI:
include/ssd_block.h): the residual addition with its RMS norm, the gated norm with an 8-bit
output, quantising in blocks of 128, the matrix product of 8-bit operands, and clipping by
the global norm of the gradients.

Like the rest of the binding this marshals arguments only; every value is computed by the
HIP kernels of libssd.so, on the current stream of the inputs' device.

8-bit operands are a ``Tensor8(q, scale)``: q holds e4m3 values, the last axis (the one that a
product sums over) padded with zeros to whole blocks of 128; scale is [blocks, rows] fp32, or
[blocks, ceil(rows / 128)] where 128 x 128 values share one.
"""
from __future__ import annotations

import ctypes
import functools
from array import array
from typing import NamedTuple, Optional, Sequence, Tuple

import torch

from .layer import _F32, _i32, _i64, _launch, _plain, _rows, _scratch, _size, _three, ssd_gated_norm_problem, \
    ssd_strides
from .layer import _norm_problem as _gated_problem
from . import SsdArgumentError, _check, _io_code, load_library

__all__ = ["Tensor8", "ssd_block_abi_version", "ssd_add_norm_fwd", "ssd_add_norm_bwd",
           "ssd_add_norm_bwd_workspace_size", "ssd_gated_norm_fwd_8bit", "ssd_quant8", "ssd_matmul8",
           "ssd_matmul8_workspace_size", "ssd_clip_grads", "ssd_clip_grads_workspace_size",
           "make_add_norm_problem", "make_quant8_problem", "make_matmul8_problem"]

BLOCK_ABI_VERSION = 1
_E4M3 = torch.float8_e4m3fn
_IO = {torch.float32: 0, torch.bfloat16: 1}
_f64 = ctypes.c_double


class Tensor8(NamedTuple):
    """Values q * scale, one scale for each block of 128 (see the module's text)."""
    q: torch.Tensor
    scale: torch.Tensor


class ssd_add_norm_problem(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("eps", ctypes.c_float),
                ("io_dtype", _i32), ("residual_dtype", _i32), ("reserved", _i32)]


class ssd_quant8_problem(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("io_dtype", _i32), ("tile", _i32),
                ("reserved", _i64)]


class ssd_matmul8_problem(ctypes.Structure):
    _fields_ = [("rows", _i64), ("cols", _i64), ("depth", _i64), ("w_tile", _i32), ("out_dtype", _i32),
                ("reserved", _i64)]


class ssd_grad(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("out", ctypes.c_void_p), ("elements", _i64), ("dtype", _i32),
                ("out_dtype", _i32)]


class ssd_clip_options(ctypes.Structure):
    _fields_ = [("max_norm", _f64), ("eps", _f64), ("grad_scale", _f64), ("reserved", _i64)]


def declare(lib) -> None:
    """Declare the entry points of ssd_block.h on an opened library."""
    if not hasattr(lib, "ssd_block_abi_version") or lib.ssd_block_abi_version() != BLOCK_ABI_VERSION:
        raise ImportError("libssd.so has another version of the block operators (rebuild it)")
    vp, sz, ptr = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
    S, psz = ptr(ssd_strides), ptr(sz)
    Pa, Pq, Pm = ptr(ssd_add_norm_problem), ptr(ssd_quant8_problem), ptr(ssd_matmul8_problem)
    for name, args in {
            "ssd_block_abi_version": [],
            "ssd_add_norm_fwd": [Pa, vp, S] + [vp] * 7,
            "ssd_add_norm_bwd_workspace_size": [Pa, psz],
            "ssd_add_norm_bwd": [Pa] + [vp] * 8 + [sz, vp],
            "ssd_gated_norm_fwd_8bit": [ptr(ssd_gated_norm_problem), vp, vp, S, vp, vp, vp, vp],
            "ssd_quant8": [Pq, vp, S] + [vp] * 5,
            "ssd_matmul8_workspace_size": [Pm, psz],
            "ssd_matmul8": [Pm] + [vp] * 6 + [sz, vp],
            "ssd_clip_grads_workspace_size": [vp, _i64, psz],
            "ssd_clip_grads": [vp, _i64, ptr(ssd_clip_options), vp, vp, sz, vp]}.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, args


def ssd_block_abi_version() -> int:
    return int(load_library().ssd_block_abi_version())


def _io(dtype, name: str) -> int:
    if dtype not in _IO:
        raise SsdArgumentError(4, "%s must be torch.float32 or torch.bfloat16, got %s" % (name, dtype))
    return _IO[dtype]


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _new8(like, lead, depth: int, scales: int) -> Tensor8:
    """An empty operand: q [*lead, whole blocks of depth], scale [blocks, scales]."""
    kb = _blocks(depth)
    return Tensor8(like.new_empty(tuple(lead) + (kb * 128,), dtype=_E4M3), like.new_empty((kb, scales), dtype=_F32))


def _output(wanted: bool, out, name: str, like, shape, dtype, dev: int):
    """An output (the caller's, checked, or a new one) and its pointer; None, None where it is not wanted.
    `like` is on its device; a contiguous one of its shape and type is the quickest to make it from."""
    if not wanted:
        return None, None
    if out is None:
        same = like.dtype is dtype and like.shape == shape and like.is_contiguous()
        out = torch.empty_like(like) if same else like.new_empty(shape, dtype=dtype)
        return out, out.data_ptr()
    return out, _plain(out, name, dtype, shape, dev)


# ---------------------------------------------------------------- residual and norm

def make_add_norm_problem(batch, seqlen, channels, eps, io_dtype, residual_dtype) -> ssd_add_norm_problem:
    return ssd_add_norm_problem(int(batch), int(seqlen), int(channels), float(eps), int(io_dtype),
                                int(residual_dtype), 0)


@functools.lru_cache(maxsize=1024)
def _add_norm_problem(*args):
    return ctypes.byref(make_add_norm_problem(*args))


@functools.lru_cache(maxsize=1024)
def _add_norm_bwd_bytes(*args):
    return _size(load_library().ssd_add_norm_bwd_workspace_size, make_add_norm_problem(*args))


def ssd_add_norm_fwd(x: torch.Tensor, residual: Optional[torch.Tensor], weight: torch.Tensor, *,
                     eps: float = 1e-5, residual_dtype: Optional[torch.dtype] = None, want_y: bool = True,
                     want_8bit: bool = False, want_h: bool = True, out: Optional[torch.Tensor] = None,
                     h_out: Optional[torch.Tensor] = None):
    """Residual addition and RMS norm.  Returns (y, y8, h), each None where it is not wanted.

    x [batch, seqlen, channels] (strided), residual the same shape or None, weight [channels]
    fp32.  h = x + residual in the residual's dtype (residual_dtype without one, by default
    that of x) is what the next block adds to and what ssd_add_norm_bwd reads; h_out may be
    ``residual``.  y is the norm of h, in the dtype of x; y8 the same as a Tensor8 by row."""
    lib = load_library()
    shape = _three(x)
    dev, io = x.get_device(), x.dtype
    if weight is None:
        raise SsdArgumentError(1, "weight must be a GPU tensor")
    if isinstance(residual, torch.Tensor):
        if residual_dtype is not None and residual_dtype != residual.dtype:
            raise SsdArgumentError(4, "residual_dtype must be the dtype of residual")
        res = residual.dtype
    else:
        res = residual_dtype if residual_dtype is not None else io
    if not (want_y or want_8bit):
        raise SsdArgumentError(10, "want_y or want_8bit must be set")
    prob = _add_norm_problem(*shape, float(eps), _io_code(x), _io(res, "residual"))
    src = _rows(x, "x", io, shape, dev)
    rp, wp = _plain(residual, "residual", res, shape, dev), _plain(weight, "weight", _F32, (shape[2],), dev)
    y, yp = _output(want_y, out, "out", x, shape, io, dev)
    h, hp = _output(want_h, h_out, "h_out", x if residual is None else residual, shape, res, dev)
    y8, qp, sp = None, None, None
    if want_8bit:
        y8 = _new8(x, shape[:2], shape[2], shape[0] * shape[1])
        qp, sp = y8.q.data_ptr(), y8.scale.data_ptr()
    _launch(lib.ssd_add_norm_fwd, dev, prob, *src, rp, wp, hp, yp, qp, sp)
    return y, y8, h


def ssd_add_norm_bwd_workspace_size(prob: ssd_add_norm_problem) -> int:
    return _size(load_library().ssd_add_norm_bwd_workspace_size, prob)


def ssd_add_norm_bwd(h: torch.Tensor, weight: torch.Tensor, dy: torch.Tensor,
                     dh: Optional[torch.Tensor] = None, *, eps: float = 1e-5, want_dx: bool = True,
                     want_dresidual: bool = True, dresidual_out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ssd_add_norm_fwd from the h that it left, dy (its dtype is that of x) and
    dh, the gradient that comes back along the residual (the dtype of h, or None).  Returns a
    dict with dx, dresidual (dresidual_out may be ``dh``) and dweight."""
    lib = load_library()
    shape = _three(h, "h")
    dev, res = h.get_device(), h.dtype
    if weight is None:
        raise SsdArgumentError(1, "weight must be a GPU tensor")
    if not isinstance(dy, torch.Tensor):
        raise SsdArgumentError(1, "dy must be a GPU tensor")
    if not (want_dx or want_dresidual):
        raise SsdArgumentError(10, "want_dx or want_dresidual must be set")
    io = dy.dtype
    key = shape + (float(eps), _io(io, "dy"), _io_code(h))
    ptrs = (_plain(h, "h", res, shape, dev), _plain(weight, "weight", _F32, (shape[2],), dev),
            _plain(dy, "dy", io, shape, dev), _plain(dh, "dh", res, shape, dev))
    dx, dxp = _output(want_dx, None, "dx", dy, shape, io, dev)
    dres, drp = _output(want_dresidual, dresidual_out, "dresidual_out", h, shape, res, dev)
    dw = torch.empty_like(weight)
    ws, ws_bytes, held = _scratch(h, workspace, _add_norm_bwd_bytes(*key) if workspace is None else 0, dev)
    _launch(lib.ssd_add_norm_bwd, dev, _add_norm_problem(*key), *ptrs, dxp, drp, dw.data_ptr(), ws, ws_bytes)
    return {"dx": dx, "dresidual": dres, "dweight": dw}


def ssd_gated_norm_fwd_8bit(x: torch.Tensor, z: Optional[torch.Tensor], weight: torch.Tensor, *,
                            ngroups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False) -> Tensor8:
    """ssd_gated_norm_fwd with its output in 8 bits, by row (what ssd_matmul8 takes).  With
    several groups their channels have to be whole blocks of 128."""
    lib = load_library()
    shape = _three(x)
    dev, io = x.get_device(), x.dtype
    if weight is None:
        raise SsdArgumentError(1, "weight must be a GPU tensor")
    key = shape + (int(ngroups), float(eps), bool(norm_before_gate), _io_code(x))
    y8 = _new8(x, shape[:2], shape[2], shape[0] * shape[1])
    _launch(lib.ssd_gated_norm_fwd_8bit, dev, _gated_problem(*key), _plain(x, "x", io, shape, dev),
            *_rows(z, "z", io, shape, dev), _plain(weight, "weight", _F32, (shape[2],), dev), y8.q.data_ptr(),
            y8.scale.data_ptr())
    return y8


# ---------------------------------------------------------------------- quantising

def make_quant8_problem(batch, seqlen, channels, io_dtype, tile) -> ssd_quant8_problem:
    return ssd_quant8_problem(int(batch), int(seqlen), int(channels), int(io_dtype), int(bool(tile)), 0)


@functools.lru_cache(maxsize=1024)
def _quant8_problem(*args):
    return ctypes.byref(make_quant8_problem(*args))


def ssd_quant8(x: torch.Tensor, *, tile: bool = False, want_rows: bool = True,
               want_cols: bool = False) -> Tuple[Optional[Tensor8], Optional[Tensor8]]:
    """A matrix in 8 bits: (rows, cols), each a Tensor8 or None where it is not wanted.

    x [batch, seqlen, channels] (strided) or [rows, channels].  ``rows`` has its shape, with
    the channels padded; ``cols`` is transposed: [channels, batch * seqlen padded].  Without
    ``tile`` each form has a scale per row of its own and block; with it 128 x 128 values share
    one (weights), and both forms hold the same values."""
    lib = load_library()
    if isinstance(x, torch.Tensor) and x.dim() == 2:
        lead, x = x.shape[:1], x.unsqueeze(0)
    else:
        lead = x.shape[:2] if isinstance(x, torch.Tensor) else None
    shape = _three(x)
    dev = x.get_device()
    if not (want_rows or want_cols):
        raise SsdArgumentError(10, "want_rows or want_cols must be set")
    n, c = shape[0] * shape[1], shape[2]
    prob = _quant8_problem(*shape, _io_code(x), bool(tile))
    src = _rows(x, "x", x.dtype, shape, dev)
    rows = _new8(x, lead, c, _blocks(n) if tile else n) if want_rows else None
    cols = _new8(x, (c,), n, _blocks(c) if tile else c) if want_cols else None
    pair = lambda t: (None, None) if t is None else (t.q.data_ptr(), t.scale.data_ptr())
    _launch(lib.ssd_quant8, dev, prob, *src, *pair(rows), *pair(cols))
    return rows, cols


# ------------------------------------------------------------------- matrix product

def make_matmul8_problem(rows, cols, depth, w_tile, out_dtype) -> ssd_matmul8_problem:
    return ssd_matmul8_problem(int(rows), int(cols), int(depth), int(bool(w_tile)), int(out_dtype), 0)


@functools.lru_cache(maxsize=1024)
def _matmul8_problem(*args):
    prob = make_matmul8_problem(*args)
    return ctypes.byref(prob), _size(load_library().ssd_matmul8_workspace_size, prob)


def ssd_matmul8_workspace_size(prob: ssd_matmul8_problem) -> int:
    return _size(load_library().ssd_matmul8_workspace_size, prob)


def _operand(t, name: str, dev: Optional[int]):
    """(q, its shape, its pointer, scale) of an 8-bit operand."""
    if not isinstance(t, tuple) or len(t) != 2:
        raise SsdArgumentError(1, "%s must be a Tensor8" % name)
    q = t[0]
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise SsdArgumentError(1, "%s.q must be a GPU tensor" % name)
    shape = q.shape
    if len(shape) < 2 or shape[-1] % 128 != 0:
        raise SsdArgumentError(2, "%s.q must be [..., depth] with a depth padded to whole blocks of 128" % name)
    return q, shape, _plain(q, name + ".q", _E4M3, shape, q.get_device() if dev is None else dev), t[1]


def ssd_matmul8(x: Tensor8, w: Tensor8, *, out_dtype: torch.dtype = torch.bfloat16,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = x w^T of 8-bit operands.  x is by row, q [..., depth]; w is by tile or by row, q
    [cols, depth].  Returns y [..., cols] in out_dtype."""
    lib = load_library()
    xq, shape, xp, xs = _operand(x, "x", None)
    dev, depth, lead = xq.get_device(), shape[-1], tuple(shape[:-1])
    rows = shape.numel() // depth if depth else 0
    _, wshape, wp, ws = _operand(w, "w", dev)
    if len(wshape) != 2 or wshape[1] != depth:
        raise SsdArgumentError(2, "w.q must be [cols, %d], got %s" % (depth, list(wshape)))
    cols, kb = wshape[0], depth // 128
    tiles = (kb, _blocks(cols))
    tile = isinstance(ws, torch.Tensor) and ws.shape == tiles
    prob, need = _matmul8_problem(rows, cols, depth, tile, _io(out_dtype, "out_dtype"))
    xsp = _plain(xs, "x.scale", _F32, (kb, rows), dev)
    wsp = _plain(ws, "w.scale", _F32, tiles if tile else (kb, cols), dev)
    y, yp = _output(True, out, "out", xq, lead + (cols,), out_dtype, dev)
    mem, mem_bytes, held = _scratch(xq, workspace, need if workspace is None else 0, dev)
    _launch(lib.ssd_matmul8, dev, prob, xp, xsp, wp, wsp, yp, mem, mem_bytes)
    return y


# ------------------------------------------------------------------------- clipping

def _clip_list(grads, out, dev) -> array:
    """The ssd_grad entries, four words each.  (A call costs its tensors' marshalling: one look at each property.)"""
    words = []
    add, io = words.extend, _IO
    try:
        if out is None:
            for g in grads:
                kind, at = io[g.dtype], g.data_ptr()
                if g.get_device() != dev or not g.is_contiguous():
                    raise KeyError
                add((at, at, g.numel(), kind | kind << 32))
        else:
            for g, o in zip(grads, out):
                n = g.numel()
                if g.get_device() != dev or o.get_device() != dev or not g.is_contiguous() or not o.is_contiguous() \
                        or o.numel() != n:
                    raise KeyError
                add((g.data_ptr(), o.data_ptr(), n, io[g.dtype] | io[o.dtype] << 32))
        return array("q", words)
    except (AttributeError, KeyError, RuntimeError):
        pass
    for g, o in zip(grads, grads if out is None else out):
        for t, name in ((g, "grads"), (o, "out")):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or t.get_device() != dev:
                raise SsdArgumentError(1, "%s must be GPU tensors on one device" % name)
            _io(t.dtype, name)
            if not t.is_contiguous():
                raise SsdArgumentError(2, "%s must be contiguous" % name)
        if o.numel() != g.numel():
            raise SsdArgumentError(2, "out must have the sizes of grads")
    raise SsdArgumentError(1, "grads must be GPU tensors with memory of their own")


@functools.lru_cache(maxsize=1024)
def _clip_options(*args):
    return ctypes.byref(ssd_clip_options(*args, 0))


def ssd_clip_grads_workspace_size(grads: Sequence[torch.Tensor]) -> int:
    words = array("q")
    for g in grads:
        words.extend((0, 0, g.numel(), 0))
    n = ctypes.c_size_t(0)
    _check(load_library().ssd_clip_grads_workspace_size(words.buffer_info()[0], len(grads), ctypes.byref(n)))
    return int(n.value)


def ssd_clip_grads(grads: Sequence[torch.Tensor], max_norm: float, *, scale: float = 1.0, eps: float = 1e-6,
                   out: Optional[Sequence[torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Clip gradients by their global norm, in place or into ``out``.  Returns the norm, an
    fp32 tensor of no axes on their device (before clipping, after ``scale``).

    Every gradient is multiplied by scale min(1, max_norm / (norm + eps)) with norm = scale
    sqrt(sum of all squares); by ``scale`` alone where the norm that is returned is not finite, or
    with max_norm infinite.  Contiguous bf16 and fp32 tensors in any mixture; ``out`` may have other dtypes
    than ``grads`` (bf16 gradients into an optimizer's fp32 buffer)."""
    lib = load_library()
    grads = list(grads)
    if not grads:
        raise SsdArgumentError(2, "there must be at least one gradient")
    out = None if out is None else list(out)
    if out is not None and len(out) != len(grads):
        raise SsdArgumentError(2, "out must have one tensor per gradient")
    first = grads[0]
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise SsdArgumentError(1, "grads must be GPU tensors on one device")
    dev = first.get_device()
    words = _clip_list(grads, out, dev)
    norm = first.new_empty((), dtype=_F32)
    need = 0
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(lib.ssd_clip_grads_workspace_size(words.buffer_info()[0], len(grads), ctypes.byref(n)))
        need = n.value
    mem, mem_bytes, held = _scratch(first, workspace, need, dev)
    _launch(lib.ssd_clip_grads, dev, words.buffer_info()[0], len(grads),
            _clip_options(float(max_norm), float(eps), float(scale)), norm.data_ptr(), mem, mem_bytes)
    return norm
