"""Pins of the fp64 references of the operators around the scan (oracle/layer.py):
closed forms, continuation through the state, and every gradient against
central differences of the forward form."""
import itertools

import numpy as np
import pytest

from oracle import layer as ref

RNG = np.random.default_rng


def numeric(f, v, eps=1e-5):
    g = np.zeros_like(v)
    for i in np.ndindex(*v.shape):
        old = v[i]
        v[i] = old + eps
        hi = f()
        v[i] = old - eps
        lo = f()
        v[i] = old
        g[i] = (hi - lo) / (2 * eps)
    return g


def check(f, inputs, got, names):
    # central differences of an O(1) loss: truncation eps^2 = 1e-10, rounding
    # 2^-53 / eps = 1e-11, both times third derivatives and sums of order 100
    for name, v in zip(names, inputs):
        num = numeric(f, v)
        assert np.allclose(got[name], num, rtol=1e-6, atol=1e-6), name


def test_conv_by_hand():
    # one channel, width 3, weights 1, 2, 4 (oldest first), inputs 1, 3, 5 after 7, 9
    x = np.array([1.0, 3.0, 5.0]).reshape(1, 3, 1)
    w = np.array([[1.0, 2.0, 4.0]])
    init = np.array([7.0, 9.0]).reshape(1, 2, 1)
    y, fin, _ = ref.conv(x, w, np.array([0.5]), init, act=False)
    assert y.ravel().tolist() == [7 + 18 + 4 + 0.5, 9 + 2 + 12 + 0.5, 1 + 6 + 20 + 0.5]
    assert fin.ravel().tolist() == [3.0, 5.0]
    y, fin, _ = ref.conv(x[:, :1], w, None, init, act=False)   # fewer tokens than the window
    assert y.ravel().tolist() == [29.0] and fin.ravel().tolist() == [9.0, 1.0]
    y, _, _ = ref.conv(np.zeros((1, 2, 1)), w, np.array([2.0]), None)
    assert np.allclose(y, 2.0 / (1.0 + np.exp(-2.0)), rtol=1e-15)


def test_conv_continues_through_the_state():
    r = RNG(0)
    x, w, b = r.normal(size=(2, 7, 3)), r.normal(size=(3, 4)), r.normal(size=3)
    y, fin, _ = ref.conv(x, w, b)
    y1, f1, _ = ref.conv(x[:, :2], w, b)
    y2, f2, _ = ref.conv(x[:, 2:], w, b, f1)
    assert np.array_equal(np.concatenate([y1, y2], 1), y) and np.array_equal(f2, fin)


@pytest.mark.parametrize("W,L,act", [(2, 5, True), (3, 1, True), (4, 2, True), (4, 5, False)])
def test_conv_gradients(W, L, act):
    r = RNG(W)
    x, w, b = r.normal(size=(2, L, 3)), r.normal(size=(3, W)), r.normal(size=3)
    init, dy = r.normal(size=(2, W - 1, 3)), r.normal(size=(2, L, 3))
    dfin = r.normal(size=(2, W - 1, 3))

    def loss():
        y, fin, _ = ref.conv(x, w, b, init, act)
        return (y * dy).sum() + (fin * dfin).sum()
    check(loss, (x, w, b, init), ref.conv_bwd(x, w, b, init, dy, dfin, act),
          ("dx", "dweight", "dbias", "dinit"))


def test_scan_by_hand():
    # dyadic: dt A = log 2 * -1 gives a = 1/2
    ln2 = np.log(2.0)
    x = np.array([4.0, 8.0]).reshape(1, 2, 1)
    dt = np.array([1.0, 1.0]).reshape(1, 2, 1)
    A = np.array([[-ln2, 0.0]])
    B = np.array([[1.0, 2.0], [0.5, 1.0]]).reshape(1, 2, 1, 2)
    C = np.array([[1.0, 1.0], [2.0, -1.0]]).reshape(1, 2, 1, 2)
    y, fin, _, _ = ref.selscan(x, dt, A, B, C, np.array([3.0]))
    # h1 = (4, 8); h2 = (2 + 4, 8 + 8)
    assert np.allclose(y.ravel(), [12 + 12, 12 - 16 + 24], rtol=1e-15)
    assert np.allclose(fin.ravel(), [6, 16], rtol=1e-15)


def test_scan_with_one_decay_per_head_is_the_ssd_recurrence():
    import torch
    import oracle
    r = RNG(3)
    Bz, L, H, P, N = 2, 9, 2, 3, 4
    x = r.normal(size=(Bz, L, H, P)).astype(np.float32)
    dt = r.uniform(0.1, 1.0, size=(Bz, L, H)).astype(np.float32)
    A = -r.uniform(0.5, 2.0, size=H).astype(np.float32)
    B, C = (r.normal(size=(Bz, L, 1, N)).astype(np.float32) for _ in range(2))
    D = r.normal(size=H).astype(np.float32)
    t = torch.from_numpy
    y, fin, _ = oracle.recurrence(t(x), t(dt), t(A), t(B), t(C), t(D), None)
    got, h, _, _ = ref.selscan(x.reshape(Bz, L, H * P), np.repeat(dt, P, 2),
                               np.repeat(A, P)[:, None] * np.ones(N), B, C, np.repeat(D, P))
    assert np.allclose(got.reshape(y.shape), y, rtol=1e-12, atol=1e-12)
    assert np.allclose(h.reshape(fin.shape), fin, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("gate,opt", [(True, dict(softplus=True, bias=True)),
                                      (False, dict(limit=(0.2, 0.9))), (True, {})])
def test_scan_gradients(gate, opt):
    r = RNG(5)
    Bz, L, D, N, G = 2, 4, 4, 3, 2
    x, dt = r.normal(size=(Bz, L, D)), r.uniform(0.1, 1.0, size=(Bz, L, D))
    A, B, C = -r.uniform(0.5, 2, size=(D, N)), r.normal(size=(Bz, L, G, N)), r.normal(size=(Bz, L, G, N))
    Dv, z, init = r.normal(size=D), r.normal(size=(Bz, L, D)) if gate else None, r.normal(size=(Bz, D, N))
    dy, dfin = r.normal(size=(Bz, L, D)), r.normal(size=(Bz, D, N))
    opt = dict(opt)
    bias = r.normal(size=D)
    if opt.pop("bias", False):
        opt["bias"] = bias

    def loss():
        y, fin, _, _ = ref.selscan(x, dt, A, B, C, Dv, z, init, **opt)
        return (y * dy).sum() + (fin * dfin).sum()
    got = ref.selscan_bwd(x, dt, A, B, C, Dv, z, init, dy, dfin, **opt)
    check(loss, (x, dt, A, B, C, Dv, init), got, ("dx", "ddt", "dA", "dB", "dC", "dD", "dinit"))
    if gate:
        check(loss, (z,), got, ("dz",))
    if "bias" in opt:
        check(loss, (bias,), got, ("ddt_bias",))


@pytest.mark.parametrize("groups,before,gate", itertools.product((1, 3), (False, True), (False, True)))
def test_norm_gradients(groups, before, gate):
    r = RNG(7)
    x, w, dy = r.normal(size=(2, 2, 6)), r.normal(size=6), r.normal(size=(2, 2, 6))
    z = r.normal(size=(2, 2, 6)) if gate else None
    f = lambda: (ref.gated_norm(x, z, w, groups, 1e-2, before) * dy).sum()
    got = ref.gated_norm_bwd(x, z, w, dy, groups, 1e-2, before)
    check(f, (x, w), got, ("dx", "dweight"))
    if gate:
        check(f, (z,), got, ("dz",))


def test_norm_closed_form():
    # every |u| alike: the norm is the sign times the weight, up to eps
    x = np.array([3.0, -3.0, 3.0, 3.0]).reshape(1, 1, 4)
    w = np.array([1.0, 2.0, 3.0, 4.0])
    assert np.allclose(ref.gated_norm(x, None, w, 2, 0.0).ravel(), [1, -2, 3, 4], rtol=1e-15)
    assert np.array_equal(ref.gated_norm(np.zeros((1, 1, 4)), None, w).ravel(), np.zeros(4))
