"""The 64-bit definitions of the layer's calls against what the mathematics
fixes: rotations are complex products and keep scores relative, attention is
a convex combination, norms are scale-free."""

import numpy as np
import pytest

from oracle import layer


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_the_complex_product_and_passes_the_rest(interleaved):
    rng = np.random.default_rng(1)
    D, R = 64, 32
    x, ang = rng.standard_normal(D), rng.uniform(0, 6, R // 2)
    y, size = layer.rotate(x, np.concatenate([np.cos(ang), np.sin(ang)]), interleaved)
    z = x[0:R:2] + 1j * x[1:R:2] if interleaved else x[: R // 2] + 1j * x[R // 2: R]
    w = z * np.exp(1j * ang)
    got = y[0:R:2] + 1j * y[1:R:2] if interleaved else y[: R // 2] + 1j * y[R // 2: R]
    np.testing.assert_allclose(got, w, rtol=1e-13)
    np.testing.assert_array_equal(y[R:], x[R:])
    assert (size >= np.abs(y) - 1e-12).all()


def test_rotated_scores_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 64))
    freq = 10.0 ** -np.arange(32)
    turn = lambda x, p: layer.rotate(x, np.concatenate([np.cos(p * freq), np.sin(p * freq)]), False)[0]
    assert turn(q, 9) @ turn(k, 4) == pytest.approx(turn(q, 105) @ turn(k, 100), rel=1e-12)


def test_positions_count_back_from_the_length():
    assert layer.positions([0, 2, 2, 3], [5, 7, 0]) == [(0, 3), (0, 4), (2, -1)]


@pytest.mark.parametrize("window", [0, 1, 3])
def test_attention_closed_forms(window):
    rng = np.random.default_rng(3)
    k, v = rng.standard_normal((2, 9, 2, 8))
    q = np.zeros((3, 4, 8))   # equal scores: the mean of the visible values
    out, size, _, _ = layer.attention(q, k, v, 6, 1.0, window)
    for i in range(3):
        lo = 0 if not window else max(0, 6 + i - window + 1)
        for h in range(4):
            np.testing.assert_allclose(out[i, h], v[lo: 7 + i, h // 2].mean(0), rtol=1e-12)
    assert (size >= np.abs(out) - 1e-12).all()
    # a constant value is returned whatever the scores are, and scores only matter up to a shift
    q = rng.standard_normal((3, 4, 8))
    out, *_ = layer.attention(q, k, np.ones_like(v), 6, 0.3, window)
    np.testing.assert_allclose(out, 1.0, rtol=1e-12)
    # keys that a row does not see do not matter
    k2, v2 = k.copy(), v.copy()
    k2[7:], v2[7:] = np.nan, np.nan
    np.testing.assert_array_equal(layer.attention(q, k, v, 6, 0.3, window)[0][0],
                                  layer.attention(q, k2, v2, 6, 0.3, window)[0][0])


def test_attention_rows_that_see_nothing_are_zero():
    q, k = np.ones((3, 1, 8)), np.ones((1, 1, 8))
    out, *_ = layer.attention(q, k, 5 * k, -2, 1.0, 0)
    np.testing.assert_array_equal(out[:2], 0)
    np.testing.assert_array_equal(out[2], 5)


def test_block_norm_closed_forms():
    rng = np.random.default_rng(4)
    xs = [rng.standard_normal((3, 32)) for _ in range(4)]
    res, w = rng.standard_normal((3, 32)), np.ones(32)
    y, r, _ = layer.block_norm(xs, res, None, None, w, 1.0, 1.0, 0.0)
    np.testing.assert_allclose(r, res + xs[0] + xs[1] + xs[2] + xs[3], rtol=1e-12)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)
    # a normed block's size does not depend on its input's
    _, r1, _ = layer.block_norm(xs, 0 * res, w, None, w, 1.0, 0.5, 0.0)
    _, r2, _ = layer.block_norm([64 * x for x in xs], 0 * res, w, None, w, 1.0, 0.5, 0.0)
    np.testing.assert_allclose(r1, r2, rtol=1e-12)
    np.testing.assert_allclose((r1 * r1).mean(-1), 0.25, rtol=1e-12)
    # a closed gate leaves the scaled residual
    _, r, _ = layer.block_norm(xs, res, w, np.zeros((1, 32)), w, 0.75, 3.0, 1e-6)
    np.testing.assert_allclose(r, 0.75 * res, rtol=1e-12)
