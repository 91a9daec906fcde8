"""The calls around a layer of experts on the GPU, where tests/test_gpu_experts.py
does not reach: weights and gradients to their last roundings, kernels that
only some sizes take, and grids that are gone through more than once.

u = 2^-24; tolerances are derived at each test.
"""

import numpy as np
import pytest
import torch

import manifold_constrained_hyper_amd as mhc
from oracle import experts
from tests.test_gpu_experts import Guarded, U, _checked, _normal, _route, _say, _some_rows, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a HIP device")
    mhc.load()
    yield


def _within(got, want, tol, what):
    """No more than tol off, without an allowance for small numbers."""
    off = np.abs((f64(got) if isinstance(got, torch.Tensor) else got) - want)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, at {np.argwhere(bad)[:3]}, by " \
                          f"{np.max(off[bad] / np.maximum(np.abs(want[bad]), 1e-300)):.2e} of the value"


# -- choice of experts ------------------------------------------------------------------------------

def _far_logits(B, E, gen, dtype):
    """Ordinary rows, and rows whose sigmoids or shares lie below fp32's normal numbers."""
    x = torch.randn(B, E, generator=gen) * 3
    x[1::4] = -90 - 10 * torch.rand(len(x[1::4]), E, generator=gen)
    x[2::4, ::2] = 88 + 14 * torch.rand(len(x[2::4]), len(range(0, E, 2)), generator=gen)
    x[3::4, 0] = 95.0
    return x.to(dtype).cuda()


@pytest.mark.parametrize("B,E,k,groups,top_groups", [
    (40, 7, 7, 1, 1), (200, 64, 8, 8, 4), (60, 256, 16, 1, 1), (9, 1000, 32, 1, 1), (9, 1000, 8, 5, 3),
    (2600, 16, 14, 1, 1), (2603, 256, 8, 8, 4), (1100, 100, 6, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_weights_are_rounded_once(B, E, k, groups, top_groups, dtype):
    """Formed in 64 bits: exp to 2^-36, at most four of them in a weight, so 2^-33 = 2^-9 u before the one rounding
    of u (half a step of 2^-149 below the normal numbers): (1 + 2^-8) u."""
    _say(f"route weights B={B} E={E} k={k} {dtype}")
    gen = torch.Generator().manual_seed(E + k)
    x = _far_logits(B, E, gen, dtype)
    rows = np.arange(B) if B <= 200 else _some_rows(B)
    for bias in (None, _normal(gen, E, scale=0.1, dtype=torch.float32)):
        for softmax in (False, True):
            for renorm in (False, True):
                for scale in (2.5, 2.0 ** 60):
                    how = dict(groups=groups, top_groups=top_groups, softmax=softmax, renorm=renorm, scale=scale)
                    ids, weights = _route(x, k, bias, **how)
                    want, want_w = experts.route(f64(x)[rows], k, None if bias is None else f64(bias), **how)
                    assert np.array_equal(ids.cpu().numpy()[rows], want)
                    _within(f64(weights)[rows], want_w, (1 + 2.0 ** -8) * U * np.abs(want_w) + 2.0 ** -150,
                            f"weights softmax={softmax} renorm={renorm} scale={scale}")
