"""The fp64 definitions of the operators around the read step: pinned by hand values, by differences and
by differentiation (no GPU)."""

import numpy as np
import pytest

from oracle import layer


def _rope(T, rot):
    return np.arange(T)[None] + 3, (10000.0 ** (-np.arange(0, rot, 2) / rot)) if rot else None


def test_rotation_by_a_quarter_turn():
    x = np.arange(1.0, 5.0).reshape(1, 1, 1, 4)
    quarter = np.array([np.pi / 2, 0.0])
    split, _ = layer.rotate(x, np.array([[1]]), quarter, False)
    pairs, _ = layer.rotate(x, np.array([[1]]), quarter, True)
    assert np.allclose(split, [[[[-3, 2, 1, 4]]]]) and np.allclose(pairs, [[[[-2, 1, 3, 4]]]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_depends_on_distance_alone_and_keeps_lengths(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    f = _rope(1, 16)[1]
    dots = []
    for p in (0, 5, 1000):
        a, _ = layer.rotate(q, np.array([[p + 7]]), f, interleaved)
        b, _ = layer.rotate(k, np.array([[p]]), f, interleaved)
        dots.append((a * b).sum())
        assert np.isclose((a * a).sum(), (q * q).sum())
    assert np.allclose(dots, dots[0])


@pytest.mark.parametrize("norm", ["none", "rms", "l2"])
@pytest.mark.parametrize("interleaved,copies", [(False, 1), (True, 3)])
def test_norm_rope_gradient_against_differences(norm, interleaved, copies):
    rng = np.random.default_rng(2)
    B, T, H, d = 2, 3, 2, 16
    x, w = rng.standard_normal((B, T, H, d)), 1 + 0.1 * rng.standard_normal(d)
    pos, f = _rope(T, 8)
    pos = np.repeat(pos, B, 0)
    go = rng.standard_normal((B, H * copies, T, d))
    loss = lambda x, w: (layer.norm_rope(x, w, norm, 1e-3, pos, f, interleaved, copies)[0] * go).sum()  # noqa: E731
    dx, dw, _, _ = layer.norm_rope_backward(x, w, norm, 1e-3, pos, f, interleaved, go, copies)
    for _ in range(4):
        ux, uw = rng.standard_normal(x.shape), rng.standard_normal(d)
        e = 1e-6
        num = (loss(x + e * ux, w + e * uw) - loss(x - e * ux, w - e * uw)) / (2 * e)
        assert np.isclose(num, (dx * ux).sum() + (dw * uw).sum(), rtol=1e-7, atol=1e-7)


@pytest.mark.parametrize("complement", [False, True])
def test_scan_is_the_unrolled_sum(complement):
    rng = np.random.default_rng(3)
    x, g = rng.standard_normal((1, 9, 2)), -rng.random((1, 9, 2))
    h0 = rng.standard_normal((1, 2))
    hs, last, _, _ = layer.scan(x, g, h0, None, complement)
    for t in range(9):
        want = np.exp(g[0, : t + 1].sum(0)) * h0[0]
        for j in range(t + 1):
            want = want + np.exp(g[0, j + 1 : t + 1].sum(0)) * x[0, j] * ((1 - np.exp(g[0, j])) if complement else 1)
        assert np.allclose(hs[0, t], want)
    assert np.array_equal(last[0], hs[0, -1])


@pytest.mark.parametrize("complement", [False, True])
def test_scan_gradient_against_differences(complement):
    rng = np.random.default_rng(4)
    B, T, D = 2, 7, 3
    x, g, h0 = rng.standard_normal((B, T, D)), -rng.random((B, T, D)), rng.standard_normal((B, D))
    dy, dh = rng.standard_normal((B, T, D)), rng.standard_normal((B, D))
    lengths = [T, 4]

    def loss(x, g, h0):
        hs, last, _, _ = layer.scan(x, g, h0, lengths, complement)
        return np.nansum(hs * dy) + (last * dh).sum()

    dx, dg, d0 = layer.scan_backward(x, g, dy, h0, dh, lengths, complement)[:3]
    for _ in range(4):
        u = [rng.standard_normal(v.shape) for v in (x, g, h0)]
        e = 1e-6
        num = (loss(x + e * u[0], g + e * u[1], h0 + e * u[2]) - loss(x - e * u[0], g - e * u[1], h0 - e * u[2])) / (2 * e)
        assert np.isclose(num, sum((a * b).sum() for a, b in zip((dx, dg, d0), u)), rtol=1e-7, atol=1e-7)
    assert not dx[1, 4:].any() and not dg[1, 4:].any()


def test_scan_reset_drops_what_came_before():
    x = np.array([np.inf, np.nan, 2.0, 3.0]).reshape(1, 4, 1)
    g = np.array([0.0, 0.0, -np.inf, 0.0]).reshape(1, 4, 1)
    hs, last, _, _ = layer.scan(x, g, np.full((1, 1), np.nan), None, False)
    assert hs[0, 2, 0] == 2.0 and last[0, 0] == 5.0
    dx, dg, d0 = layer.scan_backward(x, g, np.ones((1, 4, 1)), None, None, None, False)[:3]
    assert dx[0, :, 0].tolist() == [2.0, 1.0, 2.0, 1.0] and dg[0, 2, 0] == 0.0


def test_beam_select_by_hand():
    third = np.log(1 / 3)
    t, p, s = layer.beam_select(np.zeros((1, 2, 3)), np.array([[0.0, 0.0]]), 4)
    assert t.tolist() == [[0, 1, 2, 0]] and p.tolist() == [[0, 0, 0, 1]] and np.allclose(s, third)
    t, p, s = layer.beam_select(np.zeros((1, 2, 3)), np.array([[-2.0, -0.5]]), 3, np.array([[0, 1]]), pad=2)
    assert t.tolist() == [[2, 0, 1]] and p.tolist() == [[1, 0, 0]] and np.allclose(s, [[-0.5, -2 + third, -2 + third]])
    t, p, s = layer.beam_select(np.array([[[np.nan, 1.0, -np.inf]]]), np.array([[-1.0]]), 3)
    assert t.tolist() == [[1, 0, 2]] and s.tolist() == [[-1.0, -np.inf, -np.inf]]


def test_beam_reorder_keeps_beams_with_a_parent_outside():
    state = np.arange(6).reshape(6, 1)
    assert layer.beam_reorder(state, np.array([[1, 1, -1], [3, 0, 2]])).ravel().tolist() == [1, 1, 2, 3, 3, 5]
