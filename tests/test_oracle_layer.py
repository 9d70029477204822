"""Pins of the layer oracle on the CPU: hand-worked values, invariants and
agreement of independent forms."""
import math

import numpy as np
import pytest

from oracle import layer as OL


def test_rms_and_layer_norm_hand_worked():
    # mean square of (3, 4, 0, 0) is 25 / 4: RMS 2.5
    y = OL.norm_rows([[3.0, 4.0, 0.0, 0.0]], [1.0, 2.0, 1.0, 1.0], None, "rms", 0.0)
    assert np.allclose(y, [[1.2, 3.2, 0.0, 0.0]], rtol=1e-15)
    # mean 2, deviations (-1, 1, -1, 1), variance 1
    y = OL.norm_rows([[1.0, 3.0, 1.0, 3.0]], np.zeros(4), np.full(4, 0.5), "layer", 0.0, offset=1.0)
    assert np.allclose(y, [[-0.5, 1.5, -0.5, 1.5]], rtol=1e-15)


def test_block_norm_composition():
    r, x = np.array([[1.0, 0.0]]), np.array([[3.0, 4.0]])
    h, y = OL.block_norm(r, x, post_weight=np.ones(2), gate=np.array([2.0, 0.5]), block_scale=2.0, residual_scale=3.0,
                         eps=0.0)
    rms = math.sqrt(12.5)
    assert np.allclose(h, [[3 + 2 * 2 * 3 / rms, 2 * 0.5 * 4 / rms]]) and y is None
    h, _ = OL.block_norm(None, x)
    assert np.array_equal(h, x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_one(interleaved):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 16))
    f = 100.0 ** (-np.arange(4) / 4)
    pos = np.array([0, 1, 7, 1000, 123456])
    y = OL.rotate(x, pos, f, interleaved)
    assert np.array_equal(y[0], x[0])                       # position 0
    assert np.array_equal(y[..., 8:], x[..., 8:])           # channels past the rotated part
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    # the product of a rotated query and key depends on their distance alone
    a = OL.rotate(x[:1], np.array([40]), f, interleaved)[0, 0, :8] @ OL.rotate(x[1:2], np.array([33]), f, interleaved)[0, 0, :8]
    b = OL.rotate(x[:1], np.array([7]), f, interleaved)[0, 0, :8] @ OL.rotate(x[1:2], np.array([0]), f, interleaved)[0, 0, :8]
    assert abs(a - b) < 1e-12
    # quarter turn: (a, b) -> (-b, a)
    q = OL.rotate(np.array([[[1.0, 2.0]]]), [1], [math.pi / 2], interleaved, magnitude=2.0)
    assert np.allclose(q, [[[-4.0, 2.0]]])


def test_row_scales():
    x = np.array([[1.0, -4.48], [0.0, 0.0], [np.inf, 1.0], [np.nan, 1.0]])
    s = OL.row_scales(x, 448.0)
    assert s[0] == 0.01 and s[1] == 1.0 and np.isnan(s[2:]).all()


def test_visible():
    assert OL.visible(2, 5, 0).tolist() == [True, True, True, True, False]
    assert OL.visible(2, 5, 1, [False, True]).tolist() == [True, True, True, False, True]
    assert OL.visible(1, 0, 0).tolist() == []
    assert OL.visible(3, 2, 0).tolist() == [False, False]   # drafted token 0 is not cached


def test_attend_one():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal(8), rng.standard_normal((6, 8)), rng.standard_normal((6, 8))
    see = np.array([1, 0, 1, 1, 0, 1], bool)
    o, lse, _ = OL.attend_one(q, k, v, 0.3, see)
    w = np.exp(0.3 * (k @ q)) * see
    assert np.allclose(o, (w @ v) / w.sum()) and np.isclose(lse, np.log(w.sum()))
    # one visible row is returned as it is; hidden rows may hold anything
    v[0] = np.nan
    o, lse, _ = OL.attend_one(q, k, v, 0.3, np.arange(6) == 4)
    assert np.allclose(o, v[4]) and np.isclose(lse, 0.3 * (k[4] @ q))
    o, lse, _ = OL.attend_one(q, k, v, 0.3, np.zeros(6, bool))
    assert not o.any() and lse == -np.inf
