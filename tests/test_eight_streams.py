"""The bound for the normalisations' gradient at n = 8 (tests/eight_streams.py)
is wide enough for 32-bit arithmetic and too narrow for a wrong iteration."""

import numpy as np
import pytest

from tests import eight_streams as e8

pytestmark = pytest.mark.cpu


@pytest.mark.parametrize("diag,spread", e8.SPREADS)
def test_arithmetic_in_32_bits(diag, spread):
    *_, dH, z = e8.inputs(diag, spread, 400, seed=1)
    z = z.astype(np.float32).astype(np.float64)
    dm = dH[:, 16:]
    most = np.abs(dm).max(1)[:, None, None]
    off = np.abs(e8.emulated(z, dm) - e8.exact(z, dm))
    assert np.all(off <= 2 * e8.U * most), np.max(off / (e8.U * most))


@pytest.mark.parametrize("diag,spread", e8.SPREADS)
def test_rounding_of_z(diag, spread):
    *_, dH, z = e8.inputs(diag, spread, 400, seed=2)
    dm = dH[:, 16:]
    most = np.abs(dm).max(1)[:, None, None]
    rng = np.random.default_rng(3)
    want = e8.exact(z, dm)
    e = 2.0 ** -20      # large against 64 bits, small against a second order
    for _ in range(8):
        moved = e8.exact(z + e * rng.choice([-1.0, 1.0], z.shape), dm)
        assert np.all(np.abs(moved - want) <= 2 * e * most)


@pytest.mark.parametrize("diag,spread", e8.SLOW)
def test_one_iteration_less_is_seen(diag, spread):
    """In most rows 19 iterations are off by more than the bound, and so is
    the sum over rows that is compared (six times the root of the sum of the
    rows' squared bounds)."""
    *_, dH, z = e8.inputs(diag, spread, 333, seed=4)
    dm = dH[:, 16:]
    off = np.abs(e8.exact(z, dm, 19) - e8.exact(z, dm)).reshape(len(z), -1).max(1)
    bound = e8.row_bound(z, dm)
    assert np.mean(off > bound) > 0.8
    total = np.abs((e8.exact(z, dm, 19) - e8.exact(z, dm)).sum(0))
    assert total.max() > 6 * np.sqrt(np.sum(bound ** 2))
