"""The distillation oracle where the unlisted ids are far below the listed: their shares of the rest
are their own softmax, whatever ln q is."""
import numpy as np
import pytest

from oracle.distill import distill


@pytest.mark.parametrize("low", [-50.0, -1e6, -1e30, -3.4028234663852886e38])
def test_the_rest_is_shared_as_the_unlisted_ids_are(low):
    z = np.full((1, 12), low)
    z[0, :3] = 1.0, 0.5, 0.0
    ids, lnt = np.array([[0, 1, 2]]), np.log(np.array([[0.5, 0.2, 0.2]]))
    o = distill(z, ids, lnt, temperature=2.0)
    e = np.exp(z[0, :3] / 2.0)
    want = np.full(12, -0.1 / 9)
    want[:3] = e / e.sum() - [0.5, 0.2, 0.2]
    # (fp64; q itself is at most 9 e^-25)
    assert np.allclose(o["grad"][0], want / 2.0, rtol=0, atol=1e-9)
    assert abs(o["grad"].sum()) < 1e-12


def test_unlisted_ids_far_below_a_listed_one():
    z = np.array([[3.4e38, 0.0, 1.0, 2.0, -1.0]])
    o = distill(z, np.array([[0]]), np.log(np.array([[0.25]])))
    e = np.exp(z[0, 1:])
    assert np.allclose(o["grad"][0], np.r_[0.75, -0.75 * e / e.sum()], rtol=0, atol=1e-15)
