"""The fp64 oracle of the calls around a layer of experts: its gradients
against differences of its forward, and its choices on cases worked by hand."""

import numpy as np
import pytest

from oracle import experts

pytestmark = pytest.mark.cpu


def _slope(f, x, d, h=1e-6):
    """The derivative of the scalar f along d, from two points."""
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


@pytest.mark.parametrize("gain", [True, False])
def test_rmsnorm_gradient(gain):
    rng = np.random.default_rng(1)
    s, dy, dsum, w = rng.normal(size=(3, 24)), rng.normal(size=(3, 24)), rng.normal(size=(3, 24)), rng.normal(size=24)
    weight = w if gain else None
    y, rstd = experts.rmsnorm(s, weight, 1e-3)
    assert np.allclose(rstd ** -2 - 1e-3, np.mean(s * s, axis=1))
    dx, dw = experts.rmsnorm_bwd(s, weight, rstd, dy, dsum)
    d = rng.normal(size=s.shape)
    want = _slope(lambda t: np.sum(dy * experts.rmsnorm(t, weight, 1e-3)[0]) + np.sum(dsum * t), s, d)
    assert abs(np.sum(dx * d) - want) < 1e-7 * np.sum(np.abs(dx * d))
    e = rng.normal(size=24)
    want = _slope(lambda t: np.sum(dy * experts.rmsnorm(s, t, 1e-3)[0]), w, e)
    assert abs(np.sum(dw * e) - want) < 1e-7 * np.sum(np.abs(dw * e))


@pytest.mark.parametrize("softmax", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient(softmax, renorm):
    rng = np.random.default_rng(2)
    x, dw = 2 * rng.normal(size=(4, 11)), rng.normal(size=(4, 5))
    x[1, 3] = -np.inf
    ids, w = experts.route(x, 5, softmax=softmax, renorm=renorm, scale=1.5)
    ids[2, 1] = -1
    ids[3, 4] = ids[3, 0]
    got = experts.route_bwd(x, ids, dw, softmax=softmax, renorm=renorm, scale=1.5)
    d = rng.normal(size=x.shape)

    def toll(t):
        return sum(np.sum(dw[b] * experts.weights_of(t[b], list(ids[b]), softmax, renorm, 1.5)) for b in range(4))

    assert abs(np.sum(got * d) - _slope(toll, x, d)) < 1e-6 * np.sum(np.abs(got * d))
    assert got[1, 3] == 0


def test_renormalised_sigmoids_far_out():
    """The weights are the scores' shares also where the scores themselves underflow."""
    w = experts.route(np.array([[-900.0, -901.0, -3e38, -2000.0]]), 2)[1]
    assert np.allclose(w, [[1 / (1 + np.exp(-1)), 1 / (1 + np.exp(1))]], rtol=1e-12)
    assert np.allclose(experts.route(np.full((1, 4), -experts.LARGEST), 3)[1], 1 / 3)


def test_choices():
    x = np.array([[0.0, 2.0, 1.0, 2.0, -np.inf, np.nan]])
    assert experts.route(x, 6)[0].tolist() == [[1, 3, 2, 0, -1, -1]]
    assert experts.route(x, 2, bias=[0, 0, 0, 0.5, 9, 9])[0].tolist() == [[3, 1]]
    # groups (0, 2), (1, 2), (-, -): by their best the first (lowest of equals)
    assert experts.route(x, 2, groups=3, top_groups=1)[0].tolist() == [[1, 0]]
    # with a bias by their two best: the second
    assert experts.route(x, 2, bias=np.zeros(6), groups=3, top_groups=1)[0].tolist() == [[3, 2]]
    ids, w = experts.route(np.full((1, 4), -np.inf), 2, softmax=True)
    assert ids.tolist() == [[-1, -1]] and w.tolist() == [[0, 0]]
    assert experts.route(np.array([[np.inf, 1.0, np.inf]]), 2, softmax=True, renorm=False)[1].tolist() == [[0.5, 0.5]]


def test_order_and_back():
    ids = np.array([[2, 0], [0, 5], [2, 2], [-1, 1]])
    slots, offsets = experts.order(ids, 4)
    assert slots.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]] and offsets.tolist() == [0, 2, 3, 6, 6]
    rng = np.random.default_rng(3)
    Y, w, g = rng.normal(size=(8, 3)), rng.normal(size=(4, 2)), rng.normal(size=(4, 3))
    out, _ = experts.combine(Y, slots, w, shared=np.ones((4, 3)))
    assert np.allclose(out[0], 1 + w[0, 0] * Y[3] + w[0, 1] * Y[0]) and np.allclose(out[3], 1 + w[3, 1] * Y[2])
    dY, dw, _ = experts.combine_bwd(Y, slots, w, g)
    assert np.isnan(dY[6:]).all() and dw[1, 1] == 0
    d = rng.normal(size=Y.shape)
    want = _slope(lambda t: np.sum(g * experts.combine(t, slots, w)[0]), Y, d)
    assert abs(np.nansum(dY * d) - want) < 1e-7
    e = rng.normal(size=w.shape)
    want = _slope(lambda t: np.sum(g * experts.combine(Y, slots, t)[0]), w, e)
    assert abs(np.sum(dw * e) - want) < 1e-7
