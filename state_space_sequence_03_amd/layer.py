"""The operators around the scan (C ABI: include/ssd_layer.h): the short causal
convolution, the selective scan and the gated group norm, each with its
gradients and its form for single tokens.

Like the rest of the binding this marshals arguments only; every value is
computed by the HIP kernels of libssd.so, on the current stream of the inputs'
device.  Operands documented as strided may be slices of wider tensors
(``proj[..., a:b]``): their last axis is contiguous, the other two may have any
stride.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple, Union

import torch

__all__ = ["ssd_layer_abi_version", "ssd_conv_fwd", "ssd_conv_step", "ssd_conv_bwd",
           "ssd_conv_bwd_workspace_size", "ssd_selscan_fwd", "ssd_selscan_step", "ssd_selscan_bwd",
           "ssd_selscan_fwd_workspace_size", "ssd_selscan_bwd_workspace_size", "ssd_gated_norm_fwd",
           "ssd_gated_norm_bwd", "ssd_gated_norm_bwd_workspace_size", "make_conv_problem",
           "make_selscan_problem", "make_gated_norm_problem"]

LAYER_ABI_VERSION = 1
_i64, _i32 = ctypes.c_int64, ctypes.c_int32


class ssd_strides(ctypes.Structure):
    _fields_ = [("batch", _i64), ("token", _i64)]


class ssd_conv_problem(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("width", _i64),
                ("nsplit", _i64), ("split", _i64 * 3), ("io_dtype", _i32), ("activation", _i32),
                ("reserved", _i64)]


class ssd_selscan_problem(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("dstate", _i64),
                ("ngroups", _i64), ("io_dtype", _i32), ("reserved", _i32)]


class ssd_gated_norm_problem(ctypes.Structure):
    _fields_ = [("batch", _i64), ("seqlen", _i64), ("channels", _i64), ("ngroups", _i64),
                ("eps", ctypes.c_float), ("norm_before_gate", _i32), ("io_dtype", _i32),
                ("reserved", _i32)]


def declare(lib, dt_transform) -> None:
    """Declare the entry points of ssd_layer.h on an opened library."""
    if not hasattr(lib, "ssd_layer_abi_version") or lib.ssd_layer_abi_version() != LAYER_ABI_VERSION:
        raise ImportError("libssd.so has another version of the layer operators (rebuild it)")
    vp, sz, ptr = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
    S, X, psz = ptr(ssd_strides), ptr(dt_transform), ptr(sz)
    Pc, Ps, Pn = ptr(ssd_conv_problem), ptr(ssd_selscan_problem), ptr(ssd_gated_norm_problem)
    scan = [vp, vp, vp, vp, S, vp, S, vp, vp, S]   # x dt A B bs C cs D z zs
    for name, args in {
            "ssd_layer_abi_version": [],
            "ssd_conv_fwd": [Pc, vp, S, vp, vp, vp, ptr(vp), vp, vp],
            "ssd_conv_step": [Pc, vp, vp, S, vp, vp, ptr(vp), vp],
            "ssd_conv_bwd_workspace_size": [Pc, psz],
            "ssd_conv_bwd": [Pc, vp, S, vp, vp, vp, ptr(vp), vp, vp, S, vp, vp, vp, vp, sz, vp],
            "ssd_selscan_fwd_workspace_size": [Ps, psz],
            "ssd_selscan_fwd": [Ps, X] + scan + [vp, vp, vp, vp, sz, vp],
            "ssd_selscan_step": [Ps, X, vp] + scan + [vp, vp],
            "ssd_selscan_bwd_workspace_size": [Ps, psz],
            "ssd_selscan_bwd": [Ps, X] + scan + [vp] * 9 + [vp, S, vp, vp, vp, sz, vp],
            "ssd_gated_norm_fwd": [Pn, vp, vp, S, vp, vp, vp],
            "ssd_gated_norm_bwd_workspace_size": [Pn, psz],
            "ssd_gated_norm_bwd": [Pn, vp, vp, S, vp, vp, vp, vp, S, vp, vp, sz, vp]}.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = ctypes.c_int, args


# The helpers of the binding's other half (tensor checks, errors, streams).
from . import SsdArgumentError, _check, _dt_transform, _io_code, load_library  # noqa: E402

_F32 = torch.float32


def ssd_layer_abi_version() -> int:
    return int(load_library().ssd_layer_abi_version())


# A call's cost is its arguments' marshalling for single tokens, so the checks
# below take one pass over a tensor's properties and say what was wrong only
# after one failed, and what depends on shapes alone (problem structs, strides,
# workspace sizes) is made once per shape.

def _plain(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int):
    """Pointer of a contiguous operand of the given type, shape and device (None for None)."""
    if t is None:
        return None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, dev)
    raise SsdArgumentError(2, "%s must be contiguous" % name)


def _refuse(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SsdArgumentError(1, "%s must be a GPU tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise SsdArgumentError(2, "%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.dtype != dtype:
        raise SsdArgumentError(4, "%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.get_device() != dev:
        raise SsdArgumentError(1, "%s must be on the device of x (cuda:%d), got %s" % (name, dev, t.device))


@functools.lru_cache(maxsize=1024)
def _strides(batch: int, token: int):
    return ctypes.byref(ssd_strides(batch, token))


def _rows(t: Optional[torch.Tensor], name: str, dtype, shape, dev: int):
    """(pointer, ssd_strides reference) of a strided operand."""
    if t is None:
        return None, None
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev:
            s = t.stride()
            inner = 1
            for i in range(len(s) - 1, 1, -1):
                if shape[i] != 1 and s[i] != inner:
                    raise SsdArgumentError(2, "%s must be contiguous beyond its first two axes" % name)
                inner *= shape[i]
            return t.data_ptr(), _strides(s[0], s[1])
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, dev)
    raise SsdArgumentError(2, "%s must be %s" % (name, list(shape)))


def _three(x, name="x"):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise SsdArgumentError(1, "%s must be a GPU tensor" % name)
    shape = x.shape
    if len(shape) != 3:
        raise SsdArgumentError(2, "%s must be [batch, seqlen, channels]" % name)
    return tuple(shape)


def _scratch(x, workspace, need: int, dev: int):
    """(pointer, bytes) of the caller's workspace or of a new one."""
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    elif not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev:
        raise SsdArgumentError(1, "workspace must be a GPU tensor on the device of x")
    elif not workspace.is_contiguous():
        raise SsdArgumentError(2, "workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _launch(fn, dev: int, *args) -> None:
    """Call an entry point on the current stream of device `dev`, with that device
    current: launches go to streams of the current device."""
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            st = fn(*args, stream)
    if st:
        _check(st)


def _size(fn, prob) -> int:
    n = ctypes.c_size_t(0)
    _check(fn(ctypes.byref(prob), ctypes.byref(n)))
    return int(n.value)


# ---------------------------------------------------------------- convolution

_ACTIVATIONS = {None: 0, "silu": 1}


def make_conv_problem(batch, seqlen, channels, width, split, io_dtype, activation) -> ssd_conv_problem:
    parts = [int(c) for c in split]
    if not 1 <= len(parts) <= 3:
        raise SsdArgumentError(2, "split must have one to three parts")
    return ssd_conv_problem(int(batch), int(seqlen), int(channels), int(width), len(parts),
                            (_i64 * 3)(*(parts + [0] * (3 - len(parts)))), int(io_dtype),
                            int(activation), 0)


@functools.lru_cache(maxsize=1024)
def _conv_problem(*args):
    return ctypes.byref(make_conv_problem(*args))


@functools.lru_cache(maxsize=1024)
def _conv_bwd_bytes(*args):
    return _size(load_library().ssd_conv_bwd_workspace_size, make_conv_problem(*args))


def _conv(x, weight, bias, activation, split):
    """(device, shape of x, width, sizes of the split, problem arguments, pointers)."""
    shape = _three(x)
    dev = x.get_device()
    if activation not in _ACTIVATIONS:
        raise SsdArgumentError(10, "activation must be None or 'silu', got %r" % (activation,))
    wshape = tuple(weight.shape) if isinstance(weight, torch.Tensor) else ()
    if len(wshape) != 2 or wshape[0] != shape[2]:
        raise SsdArgumentError(2, "weight must be [channels, width]")
    sizes = (shape[2],) if split is None else tuple(map(int, split))
    if not 1 <= len(sizes) <= 3 or sum(sizes) != shape[2] or min(sizes) < 1:
        raise SsdArgumentError(2, "split must have one to three positive parts that add up to channels, got %s"
                               % (sizes,))
    key = shape + (wshape[1], sizes, _io_code(x), _ACTIVATIONS[activation])
    ptrs = _rows(x, "x", x.dtype, shape, dev) + (_plain(weight, "weight", _F32, wshape, dev),
                                                 _plain(bias, "bias", _F32, (shape[2],), dev))
    return dev, shape, wshape[1], sizes, key, ptrs


def _conv_outputs(x, shape, sizes, split, out, dev):
    """The outputs and the array of their pointers."""
    if out is None:
        ys = [x.new_empty((shape[0], shape[1], c)) for c in sizes]
        return ys, (ctypes.c_void_p * 3)(*[t.data_ptr() for t in ys])
    ys = [out] if split is None else list(out)
    return ys, _conv_parts(ys, x, shape, sizes, "out", dev)


def _like(x, out, dev):
    """A contiguous output of the shape of x (the caller's or a new one) and its pointer."""
    if out is None:
        out = torch.empty_like(x)
        return out, out.data_ptr()
    return out, _plain(out, "out", x.dtype, x.shape, dev)


def _conv_parts(ts, x, shape, sizes, name, dev):
    if len(ts) != len(sizes):
        raise SsdArgumentError(2, "%s must have one tensor per part of the split" % name)
    return (ctypes.c_void_p * 3)(*[_plain(t, name, x.dtype, (shape[0], shape[1], c), dev)
                                   for t, c in zip(ts, sizes)])


def ssd_conv_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
                 init_state: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
                 split: Optional[Sequence[int]] = None, want_final_state: bool = False, out=None,
                 final_out: Optional[torch.Tensor] = None):
    """Short causal convolution over a prompt.  Returns (y, final_state).

    x [batch, seqlen, channels] (strided), weight [channels, width] fp32, bias [channels]
    fp32, init_state [batch, width - 1, channels]: the inputs before the first
    token.  ``split`` gives the channels of up to three outputs; y is then the list
    of them, each contiguous (what ssd_fwd takes as x, B and C after a view).
    final_state, where wanted, holds the last width - 1 inputs."""
    lib = load_library()
    dev, shape, width, sizes, key, ptrs = _conv(x, weight, bias, activation, split)
    state = (shape[0], width - 1, shape[2])
    ys, parts = _conv_outputs(x, shape, sizes, split, out, dev)
    fin = None
    if want_final_state:
        fin = final_out if final_out is not None else x.new_empty(state)
    _launch(lib.ssd_conv_fwd, dev, _conv_problem(*key), *ptrs,
            _plain(init_state, "init_state", x.dtype, state, dev),
            parts, _plain(fin, "final_out", x.dtype, state, dev))
    return (ys[0] if split is None else ys), fin


def ssd_conv_step(state: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                  bias: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
                  split: Optional[Sequence[int]] = None, out=None):
    """Advance ``state`` [batch, width - 1, channels] (io dtype, in place) through the
    seqlen tokens of x.  Returns y as ssd_conv_fwd does."""
    lib = load_library()
    dev, shape, width, sizes, key, ptrs = _conv(x, weight, bias, activation, split)
    ys, parts = _conv_outputs(x, shape, sizes, split, out, dev)
    _launch(lib.ssd_conv_step, dev, _conv_problem(*key),
            _plain(state, "state", x.dtype, (shape[0], width - 1, shape[2]), dev), *ptrs,
            parts)
    return ys[0] if split is None else ys


def ssd_conv_bwd_workspace_size(prob: ssd_conv_problem) -> int:
    return _size(load_library().ssd_conv_bwd_workspace_size, prob)


def ssd_conv_bwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor],
                 init_state: Optional[torch.Tensor],
                 dy: Union[torch.Tensor, Sequence[torch.Tensor]],
                 dfinal: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
                 want_dinit: bool = False, dx_out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ssd_conv_fwd.  dy is one tensor, or a sequence of the split's;
    dx_out (strided) may be a slice of the projection's gradient.  Returns a dict with
    dx, dweight, dbias (None without bias) and, when asked, dinit."""
    lib = load_library()
    one = isinstance(dy, torch.Tensor)
    dys = [dy] if one else list(dy)
    split = None if one else [_three(t, "dy")[2] for t in dys]
    dev, shape, width, sizes, key, ptrs = _conv(x, weight, bias, activation, split)
    state = (shape[0], width - 1, shape[2])
    parts = _conv_parts(dys, x, shape, sizes, "dy", dev)
    dx = dx_out if dx_out is not None else x.new_empty(shape)
    dw = weight.new_empty((shape[2], width))
    db = weight.new_empty((shape[2],)) if bias is not None else None
    dinit = x.new_empty(state) if want_dinit else None
    ws, ws_bytes, held = _scratch(x, workspace, _conv_bwd_bytes(*key) if workspace is None else 0, dev)
    _launch(lib.ssd_conv_bwd, dev, _conv_problem(*key), *ptrs,
            _plain(init_state, "init_state", x.dtype, state, dev), parts,
            _plain(dfinal, "dfinal", x.dtype, state, dev), *_rows(dx, "dx_out", x.dtype, shape, dev),
            dw.data_ptr(), None if db is None else db.data_ptr(),
            None if dinit is None else dinit.data_ptr(), ws, ws_bytes)
    return {"dx": dx, "dweight": dw, "dbias": db, "dinit": dinit}


# -------------------------------------------------------------- selective scan

def make_selscan_problem(batch, seqlen, channels, dstate, ngroups, io_dtype) -> ssd_selscan_problem:
    return ssd_selscan_problem(int(batch), int(seqlen), int(channels), int(dstate), int(ngroups),
                               int(io_dtype), 0)


@functools.lru_cache(maxsize=1024)
def _scan_problem(*args):
    return ctypes.byref(make_selscan_problem(*args))


@functools.lru_cache(maxsize=1024)
def _scan_bytes(backward, *args):
    lib = load_library()
    return _size(lib.ssd_selscan_bwd_workspace_size if backward else lib.ssd_selscan_fwd_workspace_size,
                 make_selscan_problem(*args))


def _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit):
    """(device, problem arguments, (transform, its reference), pointers, state's shape)."""
    shape = _three(x)
    dev, io = x.get_device(), x.dtype
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        raise SsdArgumentError(2, "B and C must be [batch, seqlen, ngroups, dstate]")
    if A is None:
        raise SsdArgumentError(1, "A must be a GPU tensor")
    G, N = B.shape[2], B.shape[3]
    key = shape + (N, G, _io_code(x))
    ch = (shape[2],)
    if dt_bias is not None:
        _plain(dt_bias, "dt_bias", _F32, ch, dev)
    xf = _dt_transform(shape[2], dt_bias, dt_softplus, dt_limit)
    bc = (shape[0], shape[1], G, N)
    ptrs = (_plain(x, "x", io, shape, dev), _plain(dt, "dt", io, shape, dev),
            _plain(A, "A", _F32, (shape[2], N), dev)) + _rows(B, "B", io, bc, dev) + \
        _rows(C, "C", io, bc, dev) + (_plain(D, "D", _F32, ch, dev),) + _rows(z, "z", io, shape, dev)
    return dev, key, xf, ptrs, (shape[0], shape[2], N)


def ssd_selscan_fwd_workspace_size(prob: ssd_selscan_problem) -> int:
    return _size(load_library().ssd_selscan_fwd_workspace_size, prob)


def ssd_selscan_fwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                    C: torch.Tensor, D: Optional[torch.Tensor] = None,
                    z: Optional[torch.Tensor] = None, init_state: Optional[torch.Tensor] = None, *,
                    want_final_state: bool = True, out: Optional[torch.Tensor] = None,
                    final_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    dt_bias: Optional[torch.Tensor] = None, dt_softplus: bool = False,
                    dt_limit: Optional[Tuple[float, float]] = None):
    """Selective scan over a prompt: a decay exp(dt A[c, n]) for every channel and state.
    Returns (y, final_state).

    x, dt [batch, seqlen, channels] io dtype; A [channels, dstate] and D [channels]
    fp32; B, C (strided) [batch, seqlen, ngroups, dstate]; z (strided), the shape of x:
    y is multiplied by z sigmoid(z); init_state [batch, channels, dstate] fp32.
    dt_bias [channels], dt_softplus, dt_limit: raw step size, as in ssd_fwd."""
    lib = load_library()
    dev, key, (xf, xfp), ptrs, state = _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    y, yp = _like(x, out, dev)
    fin = None
    if want_final_state:
        fin = final_out if final_out is not None else A.new_empty(state)
    ws, ws_bytes, held = _scratch(x, workspace, _scan_bytes(False, *key) if workspace is None else 0, dev)
    _launch(lib.ssd_selscan_fwd, dev, _scan_problem(*key), xfp, *ptrs,
            _plain(init_state, "init_state", _F32, state, dev), yp,
            _plain(fin, "final_out", _F32, state, dev), ws, ws_bytes)
    return y, fin


def ssd_selscan_step(state: torch.Tensor, x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                     B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor] = None,
                     z: Optional[torch.Tensor] = None, *, dt_bias: Optional[torch.Tensor] = None,
                     dt_softplus: bool = False, dt_limit: Optional[Tuple[float, float]] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Advance ``state`` [batch, channels, dstate] (fp32, in place) through the seqlen
    tokens of x one at a time.  Arguments as for ssd_selscan_fwd; returns y."""
    lib = load_library()
    dev, key, (xf, xfp), ptrs, shape = _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    y, yp = _like(x, out, dev)
    _launch(lib.ssd_selscan_step, dev, _scan_problem(*key), xfp, _plain(state, "state", _F32, shape, dev),
            *ptrs, yp)
    return y


def ssd_selscan_bwd_workspace_size(prob: ssd_selscan_problem) -> int:
    return _size(load_library().ssd_selscan_bwd_workspace_size, prob)


def ssd_selscan_bwd(x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                    C: torch.Tensor, D: Optional[torch.Tensor], z: Optional[torch.Tensor],
                    init_state: Optional[torch.Tensor], dy: torch.Tensor,
                    dfinal: Optional[torch.Tensor] = None, *, dt_bias: Optional[torch.Tensor] = None,
                    dt_softplus: bool = False, dt_limit: Optional[Tuple[float, float]] = None,
                    want_dinit: bool = False, want_ddt_bias: bool = False,
                    dz_out: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ssd_selscan_fwd.  Returns a dict with dx, ddt (io dtype, with respect
    to the dt argument), dA, dB, dC and, where the input or the option is there, dD, dz,
    dinit and ddt_bias (None otherwise).  dz_out (strided) may be a slice of the
    projection's gradient."""
    lib = load_library()
    dev, key, (xf, xfp), ptrs, state = _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    bc = tuple(B.shape)
    got = {"dx": torch.empty_like(x), "ddt": torch.empty_like(x), "dA": torch.empty_like(A),
           "dB": x.new_empty(bc), "dC": x.new_empty(bc), "dD": torch.empty_like(D) if D is not None else None,
           "dz": None, "dinit": A.new_empty(state) if want_dinit else None,
           "ddt_bias": A.new_empty((state[1],)) if want_ddt_bias else None}
    if z is not None:
        got["dz"] = dz_out if dz_out is not None else x.new_empty(x.shape)
    ws, ws_bytes, held = _scratch(x, workspace, _scan_bytes(True, *key) if workspace is None else 0, dev)
    ptr = lambda k: None if got[k] is None else got[k].data_ptr()
    _launch(lib.ssd_selscan_bwd, dev, _scan_problem(*key), xfp, *ptrs,
            _plain(init_state, "init_state", _F32, state, dev), _plain(dy, "dy", x.dtype, x.shape, dev),
            _plain(dfinal, "dfinal", _F32, state, dev), ptr("dx"), ptr("ddt"), ptr("dA"), ptr("dB"), ptr("dC"),
            ptr("dD"), *_rows(got["dz"], "dz_out", x.dtype, x.shape, dev), ptr("dinit"), ptr("ddt_bias"), ws,
            ws_bytes)
    return got


# ------------------------------------------------------------------ gated norm

def make_gated_norm_problem(batch, seqlen, channels, ngroups, eps, norm_before_gate,
                            io_dtype) -> ssd_gated_norm_problem:
    return ssd_gated_norm_problem(int(batch), int(seqlen), int(channels), int(ngroups), float(eps),
                                  int(bool(norm_before_gate)), int(io_dtype), 0)


@functools.lru_cache(maxsize=1024)
def _norm_problem(*args):
    return ctypes.byref(make_gated_norm_problem(*args))


@functools.lru_cache(maxsize=1024)
def _norm_bwd_bytes(*args):
    return _size(load_library().ssd_gated_norm_bwd_workspace_size, make_gated_norm_problem(*args))


def _gated_norm(x, z, weight, ngroups, eps, norm_before_gate):
    shape = _three(x)
    dev = x.get_device()
    if weight is None:
        raise SsdArgumentError(1, "weight must be a GPU tensor")
    key = shape + (int(ngroups), float(eps), bool(norm_before_gate), _io_code(x))
    return dev, shape, key, (_plain(x, "x", x.dtype, shape, dev),) + _rows(z, "z", x.dtype, shape, dev) + \
        (_plain(weight, "weight", _F32, (shape[2],), dev),)


def ssd_gated_norm_fwd(x: torch.Tensor, z: Optional[torch.Tensor], weight: torch.Tensor, *,
                       ngroups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped RMS norm with a SiLU gate.  x [batch, seqlen, channels], z (strided) the
    same shape or None, weight [channels] fp32.  The gate is applied to x, or with
    norm_before_gate to the normalised output.  Returns y."""
    lib = load_library()
    dev, shape, key, ptrs = _gated_norm(x, z, weight, ngroups, eps, norm_before_gate)
    y, yp = _like(x, out, dev)
    _launch(lib.ssd_gated_norm_fwd, dev, _norm_problem(*key), *ptrs, yp)
    return y


def ssd_gated_norm_bwd_workspace_size(prob: ssd_gated_norm_problem) -> int:
    return _size(load_library().ssd_gated_norm_bwd_workspace_size, prob)


def ssd_gated_norm_bwd(x: torch.Tensor, z: Optional[torch.Tensor], weight: torch.Tensor,
                       dy: torch.Tensor, *, ngroups: int = 1, eps: float = 1e-5,
                       norm_before_gate: bool = False, dz_out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> dict:
    """Gradients of ssd_gated_norm_fwd: a dict with dx, dz (None without z; dz_out,
    strided, may be a slice of the projection's gradient) and dweight."""
    lib = load_library()
    dev, shape, key, ptrs = _gated_norm(x, z, weight, ngroups, eps, norm_before_gate)
    dx = torch.empty_like(x)
    dz = None
    if z is not None:
        dz = dz_out if dz_out is not None else x.new_empty(x.shape)
    dw = torch.empty_like(weight)
    ws, ws_bytes, held = _scratch(x, workspace, _norm_bwd_bytes(*key) if workspace is None else 0, dev)
    _launch(lib.ssd_gated_norm_bwd, dev, _norm_problem(*key), *ptrs, _plain(dy, "dy", x.dtype, shape, dev),
            dx.data_ptr(), *_rows(dz, "dz_out", x.dtype, shape, dev), dw.data_ptr(), ws, ws_bytes)
    return {"dx": dx, "dz": dz, "dweight": dw}
