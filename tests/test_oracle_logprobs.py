"""The log-probability oracle on closed forms and hand-worked rows."""
import numpy as np

from oracle.logprobs import token_logprobs


def test_two_ids_at_odds_of_three():
    r = token_logprobs(np.array([[0.0, np.log(3.0)]]), [0], 2)
    assert np.allclose(r["logp"], np.log(0.25)) and r["top_ids"].tolist() == [[1, 0]]
    assert np.allclose(r["entropy"], -(0.25 * np.log(0.25) + 0.75 * np.log(0.75)))
    r = token_logprobs(np.array([[0.0, np.log(3.0)]]), [0], 1, 0.5)
    assert np.allclose(r["logp"], np.log(0.1))


def test_uniform_rows_and_ties():
    for v in (0.0, -3.4028234663852886e38, 7.5):
        r = token_logprobs(np.full((1, 50), v), [9], 4)
        assert np.allclose(r["logp"], -np.log(50)) and np.allclose(r["entropy"], np.log(50))
        assert r["top_ids"].tolist() == [[0, 1, 2, 3]]


def test_masked_ids_have_no_probability():
    x = np.full((2, 6), -np.inf)
    x[0, 4], x[0, 1] = 1.0, 1.0
    r = token_logprobs(x, [4, 0], 3)
    assert np.allclose(r["logp"][0], np.log(0.5)) and np.allclose(r["entropy"][0], np.log(2))
    assert r["top_ids"][0].tolist() == [1, 4, 0] and r["top_logp"][0, 2] == -np.inf
    assert r["bad"].tolist() == [False, True]


def test_shift_invariance_and_unscored_rows():
    g = np.random.default_rng(1)
    x = g.standard_normal((3, 40))
    a, b = token_logprobs(x, [1, -1, 40], 5), token_logprobs(x + 1000.0, [1, -1, 40], 5)
    assert np.allclose(a["logp"][0], b["logp"][0]) and np.isnan(a["logp"][1:]).all()
    assert (a["top_ids"][1] == -1).all() and (a["top_ids"][2] >= 0).all()
    p = np.exp(x[0] - x[0].max())
    assert np.allclose(np.exp(a["logp"][0]), (p / p.sum())[1])
