"""What the key-value cache oracle makes of infinite scores, by hand."""

import numpy as np
import pytest

import oracle

INF = float("inf")


@pytest.fixture(autouse=True)
def quiet():
    with np.errstate(all="ignore"):
        yield


def attend(k, v):
    """One head of one element a token over the keys and values given (the
    score is the key)."""
    n = len(k)
    pools = [np.array(x, dtype=np.float64).reshape(1, 1, n, 1) for x in (k, v)]
    out, _, _ = oracle.paged_attention(np.ones((1, 1, 1)), *pools, np.zeros((1, 1), int), [n], 1.0)
    return out[0, 0, 0]


def test_scores_of_minus_infinity():
    assert attend([-INF, 0.0], [7.0, 3.0]) == 3.0          # weigh 0
    assert attend([-INF, -INF], [7.0, 3.0]) == 0.0         # alone: zeros, as no token at all
    assert attend([-INF], [INF]) == 0.0
    assert np.isnan(attend([-INF, 0.0], [INF, 3.0]))       # 0 times infinity


def test_other_infinities_follow_the_formula():
    assert np.isnan(attend([INF, 0.0], [7.0, 3.0]))
    assert attend([-30.0, 0.0], [INF, 3.0]) == INF
    assert np.isnan(attend([0.0, 0.0], [INF, -INF]))
