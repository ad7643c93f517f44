"""Pins of the fp64 references of the operators of a residual block (oracle/block.py)."""
import numpy as np
import pytest
import torch

from oracle import block as ref
from test_oracle_layer import numeric

RNG = np.random.default_rng


def test_e4m3_values():
    # the format's corner values, and torch's table of the same codes
    assert ref.E4M3[0] == 0 and ref.E4M3[1] == 2.0 ** -9 and ref.E4M3[8] == 2.0 ** -6 and ref.E4M3[-1] == 448.0
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, ref.E4M3)


def test_nearest8():
    # between 16 and 18 the middle goes to the even code, as between 18 and 20
    assert ref.nearest8(np.array([17.0, 17.01, 19.0, -19.0, 448.0, 500.0])).tolist() == [16, 18, 20, -20, 448, 448]
    assert ref.nearest8(np.array([2.0 ** -10, 3 * 2.0 ** -10])).tolist() == [0.0, 2.0 ** -8]
    v = RNG(0).normal(size=4000) * 100
    v = v[np.abs(v) <= 448]
    assert np.array_equal(ref.nearest8(v.astype(np.float32)), torch.from_numpy(v.astype(np.float32)).to(
        torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("down", [1, 128])
def test_blocks(down):
    v = RNG(1).normal(size=(130, 200)) * np.exp(RNG(2).normal(size=(130, 1)))
    q, s = ref.quant(v, down)
    assert q.shape == (130, 256) and s.shape == (2, 130 if down == 1 else 2) and (q[:, 200:] == 0).all()
    back = ref.widened(q, s, down)[:, :200]
    spread = np.repeat(np.repeat(s.T, 128, 1), down, 0)[:130, :200]
    assert (np.abs(back - v) <= np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * spread) * (1 + 1e-12)).all()
    for b in range(2):
        for r in range(s.shape[1]):
            part = np.abs(v[r * down:(r + 1) * down, b * 128:(b + 1) * 128])
            assert s[b, r] == part.max() / 448.0 and np.abs(q[r * down:(r + 1) * down, b * 128:(b + 1) * 128]).max() == 448
    assert ref.quant(np.zeros((1, 5)))[0].any() == 0
    same, _ = ref.quant(v.T, 128)
    if down == 128:   # a tile's values do not depend on which way it lies
        assert np.array_equal(same[:200, :130], q[:130, :200].T)


def test_matmul_by_hand():
    x = np.zeros((1, 256)); w = np.zeros((130, 256))
    x[0, 0], x[0, 128], w[129, 0], w[129, 128] = 2, 4, 8, 16
    xs, ws = np.array([[0.5], [0.25]]), np.array([[1.0, 3.0], [1.0, 5.0]])
    y, mag = ref.matmul(x, xs, w, ws, True)
    assert y[0, 129] == 2 * 8 * 0.5 * 3 + 4 * 16 * 0.25 * 5 == mag[0, 129] and (y[0, :129] == 0).all()


def test_norm_and_gradients():
    g = RNG(3)
    h, w, dy, up = g.normal(size=(2, 3, 5)), g.normal(size=5), g.normal(size=(2, 3, 5)), g.normal(size=(2, 3, 5))
    assert np.allclose(ref.norm(np.array([[3.0, 4.0]]), np.ones(2), 0.0), np.array([[3.0, 4.0]]) / np.sqrt(12.5))
    loss = lambda: float((ref.norm(h, w) * dy).sum() + (h * up).sum())
    dh, dw, _, _ = ref.norm_bwd(h, w, dy, up)
    for v, got in ((h, dh), (w, dw)):
        assert np.allclose(got, numeric(loss, v), rtol=1e-6, atol=1e-6)


def test_gated_is_the_layer_operators_norm():
    from oracle import layer
    g = RNG(4)
    x, z, w = g.normal(size=(2, 3, 8)), g.normal(size=(2, 3, 8)), g.normal(size=8)
    for before in (False, True):
        assert np.allclose(ref.gated(x, z, w, 2, 1e-5, before), layer.gated_norm(x, z, w, 2, 1e-5, before), rtol=1e-12)
    assert np.allclose(ref.gated(x, None, w), ref.norm(x, w), rtol=1e-12)


def test_clip():
    size, out = ref.clip([np.array([3.0]), np.array([0.0, 4.0])], 1.0, eps=0.0)
    assert size == 5.0 and np.allclose(out[0], 0.6) and np.allclose(out[1], [0, 0.8])
    size, out = ref.clip([np.array([3.0, 4.0])], 10.0, scale=0.5)
    assert size == 2.5 and out[0].tolist() == [1.5, 2.0]
    size, out = ref.clip([np.array([np.inf, 1.0])], 1.0, scale=2.0)
    assert size == np.inf and out[0].tolist() == [np.inf, 2.0]
