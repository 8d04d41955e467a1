"""Pins of the fp64 oracle of the gated linear recurrence and the norms (oracle/block.py), no
GPU needed: closed forms, pieces against the whole, and every gradient against central
differences of the forward function."""
import numpy as np
import pytest

from oracle import block

EPS = 1e-5


def _glr(rng, b=2, L=7, D=3):
    x, r, i = (rng.standard_normal((b, L, D)) for _ in range(3))
    return x, r, i, -rng.uniform(0.01, 1.5, D), rng.standard_normal((b, D))


def test_glr_closed_forms():
    rng = np.random.default_rng(0)
    x, _, i, _, h0 = _glr(rng)
    # gates fully open: a = exp(A) at every step, h the geometric sum
    A = np.array([-0.5, -1.0, -2.0])
    big = np.full_like(x, 800.0)
    a, n = np.exp(A), np.arange(1, 8)
    h, last, _ = block.glr(np.ones_like(x), big, big, A)
    want = np.sqrt(1 - a * a) * (1 - a[None] ** n[:, None]) / (1 - a)
    assert np.allclose(h, want[None], rtol=1e-13)
    # a shut recurrence gate keeps the state whatever comes in
    h, last, _ = block.glr(x, -big, i, A, h0)
    assert np.array_equal(h, np.broadcast_to(h0[:, None], h.shape)) and np.array_equal(last, h0)
    # a decay of nothing leaves the gated input
    h, _, _ = block.glr(x, big, i, np.full(3, -800.0), h0)
    assert np.allclose(h, block.sigmoid(i) * x, rtol=1e-15)


def test_glr_slow_decays_keep_their_input_term():
    """1 - a^2 = 2e-10 to full precision: the variance of the input term, not 1 - round(a)^2."""
    one = np.ones((1, 1, 1))
    h, _, _ = block.glr(one, 800 * one, 800 * one, np.array([-1e-10]))
    assert abs(h[0, 0, 0] / np.sqrt(2e-10) - 1) < 1e-9


def test_glr_in_pieces():
    rng = np.random.default_rng(1)
    x, r, i, A, h0 = _glr(rng)
    whole, last, _ = block.glr(x, r, i, A, h0)
    s, parts = h0, []
    for lo, hi in ((0, 1), (1, 5), (5, 7)):
        h, s, _ = block.glr(x[:, lo:hi], r[:, lo:hi], i[:, lo:hi], A, s)
        parts.append(h)
    assert np.array_equal(np.concatenate(parts, 1), whole) and np.array_equal(s, last)


def _differences(f, args, k, step=1e-6):
    """Central differences of the scalar f(*args) by args[k]."""
    v = args[k]
    g = np.zeros_like(v)
    for at in np.ndindex(*v.shape):
        for sign in (1, -1):
            w = v.copy()
            w[at] += sign * step
            g[at] += sign * f(*args[:k], w, *args[k + 1:]) / (2 * step)
    return g


def test_glr_gradients_by_differences():
    rng = np.random.default_rng(2)
    x, r, i, A, h0 = _glr(rng)
    dh, dfinal = rng.standard_normal(x.shape), rng.standard_normal(h0.shape)

    def loss(x, r, i, A, h0):
        h, last, _ = block.glr(x, r, i, A, h0)
        return float((h * dh).sum() + (last * dfinal).sum())

    args = [x, r, i, A, h0]
    h = block.glr(*args)[0]
    got, _ = block.glr_backward(x, r, i, A, h, dh, h0, dfinal)
    for k, name in enumerate(("dx", "dr", "di", "dA", "dh0")):
        assert np.allclose(got[name], _differences(loss, args, k), rtol=1e-6, atol=1e-8), name


def test_glr_gradient_of_a_shut_gate_is_finite():
    """sigmoid(r) = 0: a = 1, beta = 0; the slope's product with it vanishes."""
    one = np.ones((1, 2, 1))
    g, _ = block.glr_backward(one, -800 * one, one, np.array([-1.0]), 0 * one, one)
    assert all(np.isfinite(v).all() for v in g.values()) and np.array_equal(g["dr"], 0 * one)


@pytest.mark.parametrize("scale", [False, True])
def test_residual_norm_and_its_gradients(scale):
    rng = np.random.default_rng(3)
    x, res, dout, dres = (rng.standard_normal((3, 5)) for _ in range(4))
    w, sc = rng.standard_normal(5), rng.standard_normal(5) if scale else None
    out, s, _, _ = block.residual_norm(x, sc, res, w, 1e-12)
    assert np.allclose(np.mean((out / w) ** 2, -1), 1, rtol=1e-9)  # each row has a mean square of 1
    assert np.array_equal(s, res + (x * sc if scale else x))
    got, _ = block.residual_norm_backward(x, sc, s, w, EPS, dout, dres)

    def loss(x, res, w, sc):
        out, s, _, _ = block.residual_norm(x, sc if scale else None, res, w, EPS)
        return float((out * dout).sum() + (s * dres).sum())

    args = [x, res, w, sc if scale else np.ones(5)]
    for k, name in enumerate(("dx", "dres", "dw") + (("dscale",) if scale else ())):
        assert np.allclose(got[name], _differences(loss, args, k), rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("groups", [1, 3])
def test_gated_norm_and_its_gradients(groups, gate_first):
    rng = np.random.default_rng(4)
    y, z, dout = (rng.standard_normal((4, 6)) for _ in range(3))
    w = rng.standard_normal(6)
    out, _ = block.gated_norm(y, z, w, groups, gate_first, EPS)
    # the groups do not see one another
    for g in range(groups):
        c = slice(g * 6 // groups, (g + 1) * 6 // groups)
        assert np.allclose(out[:, c], block.gated_norm(y[:, c], z[:, c], w[c], 1, gate_first, EPS)[0], rtol=1e-14)
    got, _ = block.gated_norm_backward(y, z, w, groups, gate_first, EPS, dout)
    loss = lambda y, z, w: float((block.gated_norm(y, z, w, groups, gate_first, EPS)[0] * dout).sum())
    for k, name in enumerate(("dy", "dz", "dw")):
        assert np.allclose(got[name], _differences(loss, [y, z, w], k), rtol=1e-6, atol=1e-8), name


def test_gated_norm_order_matters_and_closed_form():
    y, w = np.array([[3.0, 4.0]]), np.array([1.0, 2.0])
    z = np.array([[800.0, 800.0]])  # silu(z) = z
    first, _ = block.gated_norm(y, z, w, 1, True, 1e-12)
    last, _ = block.gated_norm(y, z, w, 1, False, 1e-12)
    rms = np.sqrt(12.5)
    assert np.allclose(first, [[3 / rms, 8 / rms]]) and np.allclose(last, [[2400 / rms, 6400 / rms]])


def test_planted_mistakes_move_the_oracle_beyond_its_bounds():
    """The bounds are tight enough to tell one wrong token, gate or group from rounding."""
    rng = np.random.default_rng(5)
    x, r, i, A, h0 = _glr(rng, 1, 40, 4)
    h, _, bound = block.glr(x, r, i, A, h0)
    for wrong in (block.glr(x, r, i, A, None)[0], block.glr(x, i, r, A, h0)[0], block.glr(np.roll(x, 1, 1), r, i, A, h0)[0]):
        assert np.mean(np.abs(wrong - h) > bound) > 0.2
    dh = rng.standard_normal(h.shape)
    g, e = block.glr_backward(x, r, i, A, h, dh, h0)
    w, _ = block.glr_backward(x, r, i, A, np.roll(h, 1, 1), dh, h0)
    assert np.mean(np.abs(w["dr"] - g["dr"]) > e["dr"]) > 0.9
    y, z, wt = rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), np.ones(8)
    out, bound = block.gated_norm(y, z, wt, 2, True, EPS)
    assert (np.abs(block.gated_norm(y, z, wt, 1, True, EPS)[0] - out) > bound).all()
