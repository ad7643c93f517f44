"""The operators around the scan in numpy fp64, written out from their
definitions: the short causal convolution, the selective scan and the gated
group norm, with their gradients.  Tests only; shares no code with the library.
"""
import numpy as np


def f64(t):
    if t is None:
        return None
    if hasattr(t, "detach"):
        t = t.detach().float().cpu().numpy()
    return np.asarray(t, dtype=np.float64)


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def silu(v):
    return v * sigmoid(v)


def silu_slope(v):
    s = sigmoid(v)
    return s * (1.0 + v * (1.0 - s))


# ---- convolution: x [B, L, C], w [C, W], init [B, W - 1, C] ----

def _behind(x, w, init):
    B, L, C = x.shape
    W = w.shape[1]
    head = np.zeros((B, W - 1, C)) if init is None else f64(init)
    return np.concatenate([head, x], 1)


def conv(x, w, bias=None, init=None, act=True):
    x, w = f64(x), f64(w)
    full, L, W = _behind(x, w, init), x.shape[1], w.shape[1]
    u = np.zeros_like(x) if bias is None else np.zeros_like(x) + f64(bias)
    for t in range(L):
        for k in range(W):
            u[:, t] += w[:, k] * full[:, t + k]
    return (silu(u) if act else u), full[:, L:], u


def conv_bwd(x, w, bias, init, dy, dfinal=None, act=True):
    x, w, dy = f64(x), f64(w), f64(dy)
    _, _, u = conv(x, w, bias, init, act)
    full, L, W = _behind(x, w, init), x.shape[1], w.shape[1]
    du = dy * silu_slope(u) if act else dy
    dfull, dw = np.zeros_like(full), np.zeros_like(w)
    for t in range(L):
        for k in range(W):
            dfull[:, t + k] += w[:, k] * du[:, t]
            dw[:, k] += (du[:, t] * full[:, t + k]).sum(0)
    if dfinal is not None:
        dfull[:, L:] += f64(dfinal)
    return {"dx": dfull[:, W - 1:], "dinit": dfull[:, :W - 1], "dweight": dw, "dbias": du.sum((0, 1))}


# ---- selective scan: x, dt, z [B, L, D], A [D, N], B, C [B, L, G, N] ----

def prepare_dt(dt, bias=None, softplus=False, limit=None):
    """(dt', d dt' / d dt)."""
    v = f64(dt) + (0.0 if bias is None else f64(bias))
    slope = np.ones_like(v)
    if softplus:
        slope = sigmoid(v)
        v = np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))
    if limit is not None:
        slope = np.where((v >= limit[0]) & (v <= limit[1]), slope, 0.0)
        v = np.clip(v, *limit)
    return v, slope


def _spread(t, D):
    t = f64(t)
    return np.repeat(t, D // t.shape[2], 2)


def selscan(x, dt, A, B, C, D=None, z=None, init=None, **opt):
    """(y, final state, ungated y, [states before each token and after the last])."""
    x, A = f64(x), f64(A)
    d, _ = prepare_dt(dt, **opt)
    bb, cc = _spread(B, x.shape[2]), _spread(C, x.shape[2])
    h = np.zeros((x.shape[0],) + A.shape) if init is None else f64(init).copy()
    states, s = [h], np.empty_like(x)
    for t in range(x.shape[1]):
        h = np.exp(d[:, t, :, None] * A) * h + (d[:, t] * x[:, t])[..., None] * bb[:, t]
        states.append(h)
        s[:, t] = (cc[:, t] * h).sum(-1)
    if D is not None:
        s = s + f64(D) * x
    return (s if z is None else s * silu(f64(z))), h, s, states


def selscan_bwd(x, dt, A, B, C, D, z, init, dy, dfinal=None, mag=False, **opt):
    """mag: every term with its magnitude (for non-negative x, B, C, D, init, dy and
    dfinal), the scale of rounding errors."""
    _, _, s, states = selscan(x, dt, A, B, C, D, z, init, **opt)
    x, A, dy = f64(x), f64(A), f64(dy)
    size = np.abs if mag else (lambda v: v)
    G, ch = B.shape[2], x.shape[2]
    d, slope = prepare_dt(dt, **opt)
    bb, cc = _spread(B, ch), _spread(C, ch)
    ds = dy if z is None else dy * size(silu(f64(z)))
    g = np.zeros_like(states[0]) if dfinal is None else f64(dfinal).copy()
    skip = 0.0 if D is None else f64(D)
    got = {"dx": np.empty_like(x), "ddt": np.empty_like(x), "dA": np.zeros_like(A),
           "dB": np.empty(tuple(B.shape)), "dC": np.empty(tuple(B.shape)),
           "dD": (ds * x).sum((0, 1)), "dz": None if z is None else dy * s * size(silu_slope(f64(z)))}
    by_group = lambda v: v.reshape(v.shape[0], G, ch // G, -1).sum(2)
    for t in range(x.shape[1] - 1, -1, -1):
        g = g + ds[:, t, :, None] * cc[:, t]
        a = np.exp(d[:, t, :, None] * A)
        got["dC"][:, t] = by_group(ds[:, t, :, None] * states[t + 1])
        got["dB"][:, t] = by_group((d[:, t] * x[:, t])[..., None] * g)
        q = (g * bb[:, t]).sum(-1)
        flow = a * g * states[t]
        got["dx"][:, t] = d[:, t] * q + skip * ds[:, t]
        got["ddt"][:, t] = (x[:, t] * q + (size(A) * flow).sum(-1)) * slope[:, t]
        got["dA"] += (d[:, t, :, None] * flow).sum(0)
        g = a * g
    got["dinit"], got["ddt_bias"] = g, got["ddt"].sum((0, 1))
    return got


# ---- gated group norm: x, z [B, L, D], w [D] ----

def gated_norm(x, z, w, groups=1, eps=1e-5, before=False):
    x, w = f64(x), f64(w)
    gate = 1.0 if z is None else silu(f64(z))
    u = x if before else x * gate
    v = u.reshape(u.shape[:2] + (groups, -1))
    n = (v / np.sqrt((v * v).mean(-1, keepdims=True) + eps)).reshape(u.shape)
    return w * n * gate if before else w * n


def gated_norm_bwd(x, z, w, dy, groups=1, eps=1e-5, before=False):
    x, w, dy = f64(x), f64(w), f64(dy)
    gate, slope = (1.0, 0.0) if z is None else (silu(f64(z)), silu_slope(f64(z)))
    u = x if before else x * gate
    grouped = lambda t: t.reshape(u.shape[:2] + (groups, -1))
    r = 1.0 / np.sqrt((grouped(u) ** 2).mean(-1, keepdims=True) + eps)
    n = (grouped(u) * r).reshape(u.shape)
    dn = dy * gate if before else dy
    t = grouped(dn * w)
    du = (r * t - grouped(u) * r ** 3 * (t * grouped(u)).mean(-1, keepdims=True)).reshape(u.shape)
    got = {"dx": du if before else du * gate, "dz": None, "dweight": (dn * n).sum((0, 1))}
    if z is not None:
        got["dz"] = dy * w * n * slope if before else du * x * slope
    return got
