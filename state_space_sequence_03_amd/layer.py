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

import contextlib
import ctypes
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
from . import (SsdArgumentError, _check, _dev, _dt_transform, _io_code, _stream,  # noqa: E402
               load_library)


def ssd_layer_abi_version() -> int:
    return int(load_library().ssd_layer_abi_version())


def _on(device: torch.device):
    """A context in which `device` is the current one: launches go to streams of
    the current device."""
    if device.index is None or device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _same_device(x, *tensors):
    for t in tensors:
        if t is not None and t.device != x.device:
            raise SsdArgumentError(1, "every tensor must be on the device of x (%s), got %s"
                                   % (x.device, t.device))


def _rows(t: Optional[torch.Tensor], name: str, dtype, shape):
    """(pointer, ssd_strides reference) of a strided operand."""
    if t is None:
        return None, None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SsdArgumentError(1, "%s must be a GPU tensor" % name)
    if tuple(t.shape) != tuple(shape):
        raise SsdArgumentError(2, "%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.dtype != dtype:
        raise SsdArgumentError(4, "%s must be %s, got %s" % (name, dtype, t.dtype))
    inner = 1
    for i in range(t.dim() - 1, 1, -1):
        if t.shape[i] != 1 and t.stride(i) != inner:
            raise SsdArgumentError(2, "%s must be contiguous beyond its first two axes" % name)
        inner *= t.shape[i]
    return t.data_ptr(), ctypes.byref(ssd_strides(t.stride(0), t.stride(1)))


def _plain(t: Optional[torch.Tensor], name: str, dtype, shape):
    """Pointer of a contiguous operand of the given shape."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise SsdArgumentError(2, "%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    return _dev(t, name, dtype)


def _f32(x, *shape):
    return torch.empty(shape, dtype=torch.float32, device=x.device)


def _size(fn, prob) -> int:
    n = ctypes.c_size_t(0)
    _check(fn(ctypes.byref(prob), ctypes.byref(n)))
    return int(n.value)


def _scratch(x, workspace, need):
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    return _dev(workspace, "workspace"), workspace.numel() * workspace.element_size()


def _three(x, name="x"):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise SsdArgumentError(1, "%s must be a GPU tensor" % name)
    if x.dim() != 3:
        raise SsdArgumentError(2, "%s must be [batch, seqlen, channels]" % name)
    return x.shape


# ---------------------------------------------------------------- convolution

_ACTIVATIONS = {None: 0, "silu": 1}


def make_conv_problem(batch, seqlen, channels, width, split, io_dtype, activation) -> ssd_conv_problem:
    parts = [int(c) for c in split]
    if not 1 <= len(parts) <= 3:
        raise SsdArgumentError(2, "split must have one to three parts")
    return ssd_conv_problem(int(batch), int(seqlen), int(channels), int(width), len(parts),
                            (_i64 * 3)(*(parts + [0] * (3 - len(parts)))), int(io_dtype),
                            int(activation), 0)


def _conv(x, weight, bias, activation, split):
    bsz, L, C = _three(x)
    if activation not in _ACTIVATIONS:
        raise SsdArgumentError(10, "activation must be None or 'silu', got %r" % (activation,))
    if weight.dim() != 2 or weight.shape[0] != C:
        raise SsdArgumentError(2, "weight must be [channels, width]")
    prob = make_conv_problem(bsz, L, C, weight.shape[1], (C,) if split is None else split, _io_code(x),
                             _ACTIVATIONS[activation])
    return prob, _rows(x, "x", x.dtype, x.shape), _plain(weight, "weight", torch.float32, weight.shape), \
        _plain(bias, "bias", torch.float32, (C,))


def _conv_outputs(x, split, out):
    if out is None:
        sizes = (x.shape[2],) if split is None else split
        return [torch.empty((x.shape[0], x.shape[1], int(c)), dtype=x.dtype, device=x.device) for c in sizes]
    return [out] if split is None else list(out)


def _conv_parts(ts, x, split, name):
    sizes = (x.shape[2],) if split is None else split
    if len(ts) != len(sizes):
        raise SsdArgumentError(2, "%s must have one tensor per part of the split" % name)
    _same_device(x, *ts)
    return (ctypes.c_void_p * 3)(*[_plain(t, name, x.dtype, (x.shape[0], x.shape[1], int(c)))
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
    prob, (xp, xs), wp, bp = _conv(x, weight, bias, activation, split)
    state = (x.shape[0], weight.shape[1] - 1, x.shape[2])
    ys = _conv_outputs(x, split, out)
    fin = None
    if want_final_state:
        fin = final_out if final_out is not None else torch.empty(state, dtype=x.dtype, device=x.device)
    _same_device(x, weight, bias, init_state, fin)
    args = (xp, xs, wp, bp, _plain(init_state, "init_state", x.dtype, state),
            _conv_parts(ys, x, split, "out"), _plain(fin, "final_out", x.dtype, state))
    with _on(x.device):
        _check(lib.ssd_conv_fwd(ctypes.byref(prob), *args, _stream(x.device)))
    return (ys[0] if split is None else ys), fin


def ssd_conv_step(state: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                  bias: Optional[torch.Tensor] = None, *, activation: Optional[str] = "silu",
                  split: Optional[Sequence[int]] = None, out=None):
    """Advance ``state`` [batch, width - 1, channels] (io dtype, in place) through the
    seqlen tokens of x.  Returns y as ssd_conv_fwd does."""
    lib = load_library()
    prob, (xp, xs), wp, bp = _conv(x, weight, bias, activation, split)
    ys = _conv_outputs(x, split, out)
    _same_device(x, weight, bias, state)
    sp = _plain(state, "state", x.dtype, (x.shape[0], weight.shape[1] - 1, x.shape[2]))
    parts = _conv_parts(ys, x, split, "out")
    with _on(x.device):
        _check(lib.ssd_conv_step(ctypes.byref(prob), sp, xp, xs, wp, bp, parts, _stream(x.device)))
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
    for t in dys:
        _three(t, "dy")
    split = None if one else [t.shape[2] for t in dys]
    prob, (xp, xs), wp, bp = _conv(x, weight, bias, activation, split)
    state = (x.shape[0], weight.shape[1] - 1, x.shape[2])
    parts = _conv_parts(dys, x, split, "dy")
    dx = dx_out if dx_out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = _f32(x, *weight.shape)
    db = _f32(x, x.shape[2]) if bias is not None else None
    dinit = torch.empty(state, dtype=x.dtype, device=x.device) if want_dinit else None
    _same_device(x, weight, bias, init_state, dfinal, dx, workspace)
    dxp, dxs = _rows(dx, "dx_out", x.dtype, x.shape)
    ws, ws_bytes = _scratch(x, workspace, _size(lib.ssd_conv_bwd_workspace_size, prob)
                            if workspace is None else 0)
    args = (xp, xs, wp, bp, _plain(init_state, "init_state", x.dtype, state), parts,
            _plain(dfinal, "dfinal", x.dtype, state), dxp, dxs, _dev(dw, "dweight"), _dev(db, "dbias"),
            _dev(dinit, "dinit"), ws, ws_bytes)
    with _on(x.device):
        _check(lib.ssd_conv_bwd(ctypes.byref(prob), *args, _stream(x.device)))
    return {"dx": dx, "dweight": dw, "dbias": db, "dinit": dinit}


# -------------------------------------------------------------- selective scan

def make_selscan_problem(batch, seqlen, channels, dstate, ngroups, io_dtype) -> ssd_selscan_problem:
    return ssd_selscan_problem(int(batch), int(seqlen), int(channels), int(dstate), int(ngroups),
                               int(io_dtype), 0)


def _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit):
    bsz, L, ch = _three(x)
    if not isinstance(B, torch.Tensor) or B.dim() != 4:
        raise SsdArgumentError(2, "B and C must be [batch, seqlen, ngroups, dstate]")
    G, N = B.shape[2], B.shape[3]
    prob = make_selscan_problem(bsz, L, ch, N, G, _io_code(x))
    _same_device(x, dt, A, B, C, D, z, dt_bias)
    if dt_bias is not None and tuple(dt_bias.shape) != (ch,):
        raise SsdArgumentError(2, "dt_bias must be [channels]")
    xf, xfp = _dt_transform(ch, dt_bias, dt_softplus, dt_limit)
    args = (_plain(x, "x", x.dtype, x.shape), _plain(dt, "dt", x.dtype, x.shape),
            _plain(A, "A", torch.float32, (ch, N)), *_rows(B, "B", x.dtype, (bsz, L, G, N)),
            *_rows(C, "C", x.dtype, (bsz, L, G, N)), _plain(D, "D", torch.float32, (ch,)),
            *_rows(z, "z", x.dtype, x.shape))
    return prob, (xf, xfp), args, (bsz, ch, N)


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
    prob, (xf, xfp), args, state = _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    fin = None
    if want_final_state:
        fin = final_out if final_out is not None else _f32(x, *state)
    _same_device(x, init_state, y, fin, workspace)
    if workspace is None:
        need = _size(lib.ssd_selscan_fwd_workspace_size, prob)
        ws, ws_bytes = _scratch(x, None, need) if need else (None, 0)
    else:
        ws, ws_bytes = _scratch(x, workspace, 0)
    more = (_plain(init_state, "init_state", torch.float32, state), _plain(y, "out", x.dtype, x.shape),
            _plain(fin, "final_out", torch.float32, state), ws, ws_bytes)
    with _on(x.device):
        _check(lib.ssd_selscan_fwd(ctypes.byref(prob), xfp, *args, *more, _stream(x.device)))
    return y, fin


def ssd_selscan_step(state: torch.Tensor, x: torch.Tensor, dt: torch.Tensor, A: torch.Tensor,
                     B: torch.Tensor, C: torch.Tensor, D: Optional[torch.Tensor] = None,
                     z: Optional[torch.Tensor] = None, *, dt_bias: Optional[torch.Tensor] = None,
                     dt_softplus: bool = False, dt_limit: Optional[Tuple[float, float]] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Advance ``state`` [batch, channels, dstate] (fp32, in place) through the seqlen
    tokens of x one at a time.  Arguments as for ssd_selscan_fwd; returns y."""
    lib = load_library()
    prob, (xf, xfp), args, shape = _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_device(x, state, y)
    sp, yp = _plain(state, "state", torch.float32, shape), _plain(y, "out", x.dtype, x.shape)
    with _on(x.device):
        _check(lib.ssd_selscan_step(ctypes.byref(prob), xfp, sp, *args, yp, _stream(x.device)))
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
    prob, (xf, xfp), args, state = _selscan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, dt_limit)
    like = dict(dtype=x.dtype, device=x.device)
    got = {"dx": torch.empty(x.shape, **like), "ddt": torch.empty(x.shape, **like),
           "dA": _f32(x, *A.shape), "dB": torch.empty(B.shape, **like),
           "dC": torch.empty(B.shape, **like), "dD": _f32(x, x.shape[2]) if D is not None else None,
           "dz": None, "dinit": _f32(x, *state) if want_dinit else None,
           "ddt_bias": _f32(x, x.shape[2]) if want_ddt_bias else None}
    if z is not None:
        got["dz"] = dz_out if dz_out is not None else torch.empty(x.shape, **like)
    _same_device(x, init_state, dy, dfinal, got["dz"], workspace)
    ws, ws_bytes = _scratch(x, workspace, _size(lib.ssd_selscan_bwd_workspace_size, prob)
                            if workspace is None else 0)
    more = (_plain(init_state, "init_state", torch.float32, state), _plain(dy, "dy", x.dtype, x.shape),
            _plain(dfinal, "dfinal", torch.float32, state),
            *[_dev(got[k], k) for k in ("dx", "ddt", "dA", "dB", "dC", "dD")],
            *_rows(got["dz"], "dz_out", x.dtype, x.shape), _dev(got["dinit"], "dinit"),
            _dev(got["ddt_bias"], "ddt_bias"), ws, ws_bytes)
    with _on(x.device):
        _check(lib.ssd_selscan_bwd(ctypes.byref(prob), xfp, *args, *more, _stream(x.device)))
    return got


# ------------------------------------------------------------------ gated norm

def make_gated_norm_problem(batch, seqlen, channels, ngroups, eps, norm_before_gate,
                            io_dtype) -> ssd_gated_norm_problem:
    return ssd_gated_norm_problem(int(batch), int(seqlen), int(channels), int(ngroups), float(eps),
                                  int(bool(norm_before_gate)), int(io_dtype), 0)


def _gated_norm(x, z, weight, ngroups, eps, norm_before_gate):
    bsz, L, ch = _three(x)
    prob = make_gated_norm_problem(bsz, L, ch, ngroups, eps, norm_before_gate, _io_code(x))
    _same_device(x, z, weight)
    return prob, (_plain(x, "x", x.dtype, x.shape), *_rows(z, "z", x.dtype, x.shape),
                  _plain(weight, "weight", torch.float32, (ch,)))


def ssd_gated_norm_fwd(x: torch.Tensor, z: Optional[torch.Tensor], weight: torch.Tensor, *,
                       ngroups: int = 1, eps: float = 1e-5, norm_before_gate: bool = False,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped RMS norm with a SiLU gate.  x [batch, seqlen, channels], z (strided) the
    same shape or None, weight [channels] fp32.  The gate is applied to x, or with
    norm_before_gate to the normalised output.  Returns y."""
    lib = load_library()
    prob, args = _gated_norm(x, z, weight, ngroups, eps, norm_before_gate)
    y = out if out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_device(x, y)
    yp = _plain(y, "out", x.dtype, x.shape)
    with _on(x.device):
        _check(lib.ssd_gated_norm_fwd(ctypes.byref(prob), *args, yp, _stream(x.device)))
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
    prob, args = _gated_norm(x, z, weight, ngroups, eps, norm_before_gate)
    dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dz = None
    if z is not None:
        dz = dz_out if dz_out is not None else torch.empty(x.shape, dtype=x.dtype, device=x.device)
    dw = _f32(x, x.shape[2])
    _same_device(x, dy, dz, workspace)
    ws, ws_bytes = _scratch(x, workspace, _size(lib.ssd_gated_norm_bwd_workspace_size, prob)
                            if workspace is None else 0)
    more = (_plain(dy, "dy", x.dtype, x.shape), _dev(dx, "dx"), *_rows(dz, "dz_out", x.dtype, x.shape),
            _dev(dw, "dweight"), ws, ws_bytes)
    with _on(x.device):
        _check(lib.ssd_gated_norm_bwd(ctypes.byref(prob), *args, *more, _stream(x.device)))
    return {"dx": dx, "dz": dz, "dweight": dw}
