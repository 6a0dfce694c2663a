"""The bound of the shared-prefix decode's long cases sees a tile of 128
positions that is left out (float64 on the CPU)."""
import numpy as np
import pytest

from tests import _prefix_bound as bound


@pytest.mark.parametrize("n", [500, 2900, 5003])
def test_a_lost_tile_shows_in_every_row(n):
    rng = np.random.default_rng(n)
    k, v = rng.standard_normal((2, n, 128))
    for row in range(24):
        q = rng.standard_normal(128)
        o, err = bound.row_bound(q, k, v)
        lost = 128 * int(rng.integers(0, -(-n // 128)))
        rest = np.r_[0:lost, min(n, lost + 128):n]
        if n - lost < 128:
            continue                                 # a partial last tile
        got, _ = bound.row_bound(q, k[rest], v[rest])
        assert (np.abs(got - o) > bound.rounded(o, err)).any(), (row, lost)


def test_the_roundings_stay_inside():
    """K', V', p and the output rounded as the kernel rounds them."""
    rng = np.random.default_rng(1)
    n, d = 700, 128
    k, v = rng.standard_normal((2, n, d))
    k[:, 3] *= 8
    k[:2] *= 6
    kr, vr = (x.astype(np.float16).astype(np.float64) for x in (k, v))
    for _ in range(24):
        q = rng.standard_normal(d)
        o, err = bound.row_bound(q, k, v)
        z = kr @ q / np.sqrt(d)
        p = np.exp(z - z.max())
        got = (256 * p).astype(np.float16).astype(np.float64) / 256 @ vr / p.sum()
        assert (np.abs(got - o) <= err).all()
