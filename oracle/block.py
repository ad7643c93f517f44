"""The operators of a residual block in numpy fp64, written out from their definitions:
residual addition with RMS norm and its gradients, 8-bit values in blocks, products of them,
clipping by the global norm.  Tests only; shares no code with the library.
"""
import numpy as np

from .layer import f64, silu

MOST, LEAST = 448.0, 2.0 ** -100

# Every non-negative finite e4m3 value: 4 exponent bits (bias 7), 3 mantissa bits, no infinities.
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest8(v):
    """The e4m3 value nearest to each of v, ties to the even code; magnitudes past the largest go to it."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(v)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    low, high = E4M3[hi - 1], E4M3[hi]
    up = (a - low > high - a) | ((a - low == high - a) & (hi % 2 == 0))
    return np.where(np.isnan(v), np.nan, np.copysign(np.where(up, high, low), v))


def blocks(v, down=1):
    """v [rows, depth] in blocks of `down` rows x 128: (v * 448 / m padded to whole blocks,
    scale [blocks, rows / down], m spread over v's padded shape)."""
    v = f64(v)
    rows, depth = v.shape
    nb, nr = -(-depth // 128), -(-rows // down)
    room = np.zeros((nr * down, nb * 128))
    room[:rows, :depth] = v
    cut = np.abs(room.reshape(nr, down, nb, 128))
    m = np.maximum(np.fmax.reduce(cut, axis=(1, 3)), LEAST)
    wide = np.repeat(np.repeat(m, 128, 1), down, 0)[:rows]
    with np.errstate(invalid="ignore"):
        return room[:rows] * (MOST / wide), (m / MOST).T, wide


def quant(v, down=1):
    scaled, scale, _ = blocks(v, down)
    return nearest8(scaled), scale


def widened(q, scale, down=1):
    """The values that an 8-bit operand stands for, padding included."""
    q = f64(q)
    return q * np.repeat(np.repeat(f64(scale).T, 128, 1), down, 0)[:q.shape[0]]


def matmul(x, xs, w, ws, tile):
    a, b = widened(x, xs), widened(w, ws, 128 if tile else 1)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def norm(h, w, eps=1e-5):
    h, w = f64(h), f64(w)
    return w * h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)


def gated(x, z, w, ngroups=1, eps=1e-5, before=False):
    x, w = f64(x), f64(w)
    gate = 1.0 if z is None else silu(f64(z))
    u = x if before else x * gate
    g = u.reshape(u.shape[:-1] + (ngroups, -1))
    n = (g / np.sqrt((g * g).mean(-1, keepdims=True) + eps)).reshape(u.shape) * w
    return n * gate if before else n


def norm_bwd(h, w, dy, dh=None, eps=1e-5):
    """(dh', dw, magnitudes of the terms of each)."""
    h, w, dy = f64(h), f64(w), f64(dy)
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    n, t = h * r, dy * w
    up = 0.0 if dh is None else f64(dh)
    got = up + r * (t - n * (t * n).mean(-1, keepdims=True))
    mag = np.abs(up) + r * (np.abs(t) + np.abs(n) * np.abs(t * n).mean(-1, keepdims=True))
    lead = tuple(range(h.ndim - 1))
    return got, (dy * n).sum(lead), mag, np.abs(dy * n).sum(lead)


def clip(grads, most, scale=1.0, eps=1e-6):
    total = sum(float((f64(g) ** 2).sum()) for g in grads)
    size = scale * np.sqrt(total)
    by = scale * min(1.0, most / (size + eps)) if np.isfinite(size) else scale
    return size, [f64(g) * by for g in grads]
