"""The fp64 gradient oracle against differences of the forward oracle, and the
checkpoint oracle against the format's definition.

Central differences with step h have an error of O(h^2) third derivatives plus
rounding 2^-53 |loss| / h; at h = 1e-5 and a loss of order 10 both are below
1e-9, so gradients of order 1e-3 and more are compared to 1e-6 of the largest
one."""

import numpy as np
import pytest

import oracle
from oracle import backward

pytestmark = pytest.mark.cpu

STEP = 1e-5


def _setup(n, C, B, seed):
    rng = np.random.default_rng(seed)
    N = n * n + 2 * n
    p = {"x": rng.standard_normal((B, n * C)), "phi": rng.standard_normal((n * C, N)) / np.sqrt(n * C),
         "f_out": rng.standard_normal((B, C)), "alpha": np.array([0.7, -0.4, 0.9]),
         "b_pre": 0.3 * rng.standard_normal(n), "b_post": 0.3 * rng.standard_normal(n),
         "b_res": (2 * np.eye(n)).reshape(-1) + 0.3 * rng.standard_normal(n * n)}
    g = {"dX_next": rng.standard_normal((B, n * C)), "dF_pre": rng.standard_normal((B, C))}
    return p, g


def _forward(p, n, C):
    return oracle.forward(p["x"], p["phi"], *p["alpha"], p["b_pre"], p["b_post"], p["b_res"], p["f_out"], n, C)


def _loss(p, g, n, C):
    """A loss whose gradients with respect to X_next and F_pre are g's."""
    o = _forward(p, n, C)
    return float(np.sum(g["dX_next"] * o["X_next"]) + np.sum(g["dF_pre"] * o["F_pre"]))


def _gradients(p, g, n, C):
    o = _forward(p, n, C)
    dF_out, dH = backward.post_res_bwd(p["x"], p["f_out"], o["H"], g["dX_next"], n, C)
    d = backward.coeffs_pre_bwd(p["x"], p["phi"], p["alpha"], (p["b_pre"], p["b_post"], p["b_res"]), o["logits"],
                                o["r"], o["H"], g["dX_next"], dH, g["dF_pre"], n, C)
    return {"x": d["dX"], "phi": d["dphi"], "alpha": d["dalpha"], "f_out": dF_out,
            "b_pre": d["db_pre"], "b_post": d["db_post"], "b_res": d["db_res"]}


@pytest.mark.parametrize("n,C,B", [(1, 8, 2), (2, 8, 3), (4, 8, 2), (8, 8, 1)])
def test_gradients_against_differences(n, C, B):
    p, g = _setup(n, C, B, seed=100 * n + B)
    grads = _gradients(p, g, n, C)
    rng = np.random.default_rng(7)
    for name, got in grads.items():
        flat = p[name].reshape(-1)
        where = rng.permutation(flat.size)[:40]
        diff = np.zeros(len(where))
        for k, at in enumerate(where):
            kept = flat[at]
            flat[at] = kept + STEP
            up = _loss(p, g, n, C)
            flat[at] = kept - STEP
            down = _loss(p, g, n, C)
            flat[at] = kept
            diff[k] = (up - down) / (2 * STEP)
        want = got.reshape(-1)[where]
        assert np.max(np.abs(diff - want)) <= 1e-6 * max(1.0, np.max(np.abs(got))), name


def test_one_stream_normalises_to_nothing():
    """At n = 1 H_res is exactly 1 whatever the logit: no gradient."""
    d = backward.sinkhorn_bwd(np.array([[[0.3]], [[-4.0]]]), np.array([[[2.0]], [[5.0]]]))
    assert np.array_equal(d, np.zeros((2, 1, 1)))


def test_checkpoint_by_hand():
    """One block: the scale is the least power of two with |x| <= 448 scale."""
    x = np.zeros((1, 32))
    x[0, :4] = [448.0, -1.0, 2.0 ** -9, 3 * 2.0 ** -11]
    codes, scales = backward.ckpt_encode(x, 1, 32)
    assert scales[0, 0] == 127
    assert list(codes[0, :4]) == [0x7E, 0x80 | 0x38, 0x01, 0x01]
    x[0, 0] = 450.0                       # past 448: the scale doubles
    codes, scales = backward.ckpt_encode(x, 1, 32)
    assert scales[0, 0] == 128
    assert backward.ckpt_decode(codes, scales, 1, 32)[0, 0] == 448.0    # 225 rounds to 224
    x[0, 0] = np.inf                      # not finite: NaN, and no say in the scale
    codes, scales = backward.ckpt_encode(x, 1, 32)
    assert codes[0, 0] == 0x7F and scales[0, 0] == 119                  # 1 <= 448 * 2^-8


@pytest.mark.parametrize("C", [8, 32, 40, 100])
def test_checkpoint_error_bound(C):
    rng = np.random.default_rng(C)
    x = rng.standard_t(4, (5, 2 * C)) * np.exp2(rng.integers(-20, 20, (5, 1)))
    codes, scales = backward.ckpt_encode(x, 2, C)
    y = backward.ckpt_decode(codes, scales, 2, C)
    step = np.repeat(np.exp2(scales.reshape(5, 2, -1) - 127.0), 32, axis=2)[:, :, :C].reshape(5, 2 * C)
    assert np.all(np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, step * 2.0 ** -10))


def test_embedding_by_hand():
    table = np.arange(12.0).reshape(3, 4)
    out = backward.embed([2, -1, 0, 3], table, 0.5, 2)
    assert np.array_equal(out[0], np.tile(table[2] / 2, 2)) and not out[1].any() and not out[3].any()
    d = backward.embed_bwd([2, -1, 2, 3], np.ones((4, 8)), 0.5, 2, 4, 3)
    assert np.array_equal(d, np.array([[0.0] * 4, [0.0] * 4, [2.0] * 4]))
