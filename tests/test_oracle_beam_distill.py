"""Pins of the beam search and distillation oracles: brute force, and gradients
against central differences."""
import itertools

import numpy as np
import pytest

from oracle.beam import beam_reorder, beam_select
from oracle.distill import distill


def test_beams_of_full_width_are_exhaustive_search():
    # with every prefix kept, two steps give the best of all pairs
    r = np.random.default_rng(0)
    K = 5
    first, second = r.normal(size=K), r.normal(size=(K, K))
    ln = lambda x: x - np.log(np.exp(x).sum(-1, keepdims=True))  # noqa: E731
    one = beam_select(first[None, None], np.zeros((1, 1)), K)
    two = beam_select(second[one["tokens"][0]][None], one["scores"], 7)
    every = sorted(((ln(first)[i] + ln(second)[i, j], i, j) for i, j in itertools.product(range(K), range(K))),
                   reverse=True)[:7]
    assert np.allclose(two["scores"][0], [e[0] for e in every], atol=1e-12)
    assert [(one["tokens"][0][p], t) for p, t in zip(two["parent"][0], two["tokens"][0])] == [e[1:] for e in every]


def test_ties_ends_and_missing_beams():
    same = np.zeros((1, 3, 4))
    o = beam_select(same, np.zeros((1, 3)), 6)
    assert o["parent"][0].tolist() == [0, 0, 0, 0, 1, 1] and o["tokens"][0].tolist() == [0, 1, 2, 3, 0, 1]
    o = beam_select(same, np.array([[-np.inf, -1.0, -0.5]]), 8, done=np.array([[0, 0, 1]]), end_id=2)
    assert o["parent"][0].tolist() == [2, 1, 1, 1, 1, -1, -1, -1]
    assert o["tokens"][0].tolist() == [2, 0, 1, 2, 3, -1, -1, -1]
    assert o["done"][0].tolist() == [True, False, False, True, False, False, False, False]
    masked = np.full((1, 1, 3), -np.inf)
    assert (beam_select(masked, np.zeros((1, 1)), 2)["parent"] == -1).all()


def test_reorder_moves_positions_below_the_length():
    s = np.arange(2 * 3 * 4).reshape(2, 3, 4)
    o = beam_reorder(s, np.array([[2, -1, 0], [1, 1, 1]]), np.zeros_like(s), lengths=np.array([2, 0]), len_dim=2)
    assert o[0].tolist() == [[8, 9, 0, 0], [0, 0, 0, 0], [0, 1, 0, 0]] and not o[1].any()


@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("T", [0.5, 1.0, 3.0])
def test_gradient_is_that_of_the_loss(rest, T):
    r = np.random.default_rng(1)
    R, K, k = 4, 11, 4
    z = r.normal(size=(R, K)) * 2
    inv = np.concatenate([r.permutation(K), [-1, -1, -1]])
    ids = np.stack([r.permutation(K + 3)[:k] for _ in range(R)])
    lnt = np.log(r.dirichlet(np.ones(k + 1), R)[:, :k])
    ids[1, 2] = -1
    z[2, 5] = -np.inf
    w = r.normal(size=R)
    o = distill(z, ids, lnt, inv, rest, T, w)
    h = 1e-5
    for i in range(R):
        for j in range(K):
            if z[i, j] == -np.inf:
                assert o["grad"][i, j] == 0.0
                continue
            e = np.zeros_like(z)
            e[i, j] = h
            d = (distill(z + e, ids, lnt, inv, rest, T)["loss"][i]
                 - distill(z - e, ids, lnt, inv, rest, T)["loss"][i]) / (2 * h)
            # truncation h^2 / T^3 (at most 8e-10) and cancellation 4 eps / h (9e-11, times the loss below 20)
            assert abs(d * w[i] - o["grad"][i, j]) < 1e-8
    assert np.allclose(o["grad"].sum(1), 0.0, atol=1e-12)


def test_loss_is_a_divergence():
    r = np.random.default_rng(2)
    z = r.normal(size=(1, 9))
    p = np.exp(z - np.log(np.exp(z).sum()))
    ids = np.argsort(-z, 1)[:, :4]
    lnt = np.log(np.take_along_axis(p, ids, 1))
    assert abs(distill(z, ids, lnt)["loss"][0]) < 1e-14           # the drafter is the teacher
    assert np.abs(distill(z, ids, lnt)["grad"]).max() < 1e-15
    other = r.normal(size=(1, 9))
    for rest in (True, False):
        assert distill(other, ids, lnt, rest=rest)["loss"][0] > 0
    # nothing listed, nothing kept
    assert distill(z, np.full((1, 4), -1), lnt)["loss"][0] == 0.0
    assert distill(z, ids, np.full((1, 4), -np.inf), rest=False)["loss"][0] == 0.0
