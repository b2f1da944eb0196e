"""Pins of the beam oracle where scores are equal: the order that the interface
states, taken in whole numbers."""

import numpy as np
import pytest

from oracle import beam as ref


def in_whole_numbers(x, scores, W):
    """Beams that share one row x of whole numbers (so that the logarithm is common): the W best
    (token, beam) by score, then beam, then logit, then id."""
    x, scores = [int(v) for v in x], [int(v) for v in scores]
    every = [(-(s + v), w, -v, i) for w, s in enumerate(scores) for i, v in enumerate(x)]
    return [(i, w) for _, w, _, i in sorted(every)[:W]]


def picked(got, b, W):
    return list(zip(got[0][b].tolist(), (got[1].reshape(-1, W)[b] - b * W).tolist()))


def test_the_lower_beam_comes_first():
    x = np.full((1, 2, 9), -1.0)
    x[..., 0] = 0.0
    got = ref.beam_select(x, np.array([[-1.0, -2.0]]))
    assert picked(got, 0, 2) == [(0, 0), (1, 0)]


@pytest.mark.parametrize("seed", range(20))
def test_shared_rows(seed):
    rng = np.random.default_rng(seed)
    W = 4
    x, scores = -rng.permutation(50), rng.integers(-6, 0, W)
    got = ref.beam_select(np.tile(x.astype(float), (1, W, 1)), scores[None].astype(float))
    assert picked(got, 0, W) == in_whole_numbers(x, scores, W)


@pytest.mark.parametrize("finished_first", [True, False])
def test_finished_beside_live(finished_first):
    """A live beam with one id left has it at its own score."""
    x = np.full((1, 2, 5), -np.inf)
    x[..., 3] = 4.0
    done = np.array([[1, 0]] if finished_first else [[0, 1]])
    got = ref.beam_select(x, np.full((1, 2), -2.0), done, end=1)
    assert picked(got, 0, 2) == ([(1, 0), (3, 1)] if finished_first else [(3, 0), (1, 1)])


def test_logits_decide_within_a_beam():
    """1e-30 and 0 are equal beside a largest logit of 5, as scores."""
    x = np.full((1, 3, 20), -np.inf)
    x[0, 0, [2, 5, 10, 11]] = 5.0, 0.0, 1e-30, -0.0
    got = ref.beam_select(x, np.array([[-1.0, -np.inf, -np.inf]]))
    assert picked(got, 0, 3) == [(2, 0), (10, 0), (5, 0)]
