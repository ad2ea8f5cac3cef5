"""Routing in groups with masked experts: runs with any number of live experts, none among them, against the definition
in 64 bits (weights: rounded to f32 from a value evaluated in f64, a relative 2^-24; 2^-23 leaves room for the f64 steps)."""
import numpy as np
import pytest

import route_reference as RR
import w4_reference as R
from test_route_gpu import run

pytestmark = pytest.mark.gpu


def check(logits, k, bf16=False, **kw):
    ids, w = run(logits, k, bf16, **kw)
    if bf16:
        logits = R.bf16_values(R.bf16_bits(logits)).astype(np.float32).reshape(logits.shape)
    rid, rw = RR.route(logits, k, **kw)
    assert np.array_equal(ids, rid)
    assert (np.abs(w - rw) <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149).all()
    return ids, w


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("best", [1, 2])
def test_one_live_expert_beside_a_masked_run(score, best):
    """The live expert is chosen, whichever run it is in and whatever the masked ones' biases are."""
    inf = np.inf
    l = np.array([[-inf, -inf, -inf, 3], [-inf, -inf, 5, -inf], [np.nan, 2, -inf, np.nan], [-inf, -inf, np.nan, -1e30]], np.float32)
    for bias in (None, np.array([9, -9, 9, -9], np.float32)):
        ids, w = check(l, 1, score=score, groups=2, group_best=best, bias=bias, renormalize=score == 0)
        assert ids[:, 0].tolist() == [3, 2, 1, 3]
    l = np.array([[-5, -5, 4, -inf], [1, 1, 1.2, -inf], [-inf, 0.1, -inf, -inf]], np.float32)
    ids, _ = check(l, 1, score=score, groups=2, group_best=best)
    assert ids[0, 0] == 2 and ids[2, 0] == 1


CASES = [  # E, groups, top_groups, k
    (4, 2, 1, 1), (6, 3, 2, 4), (64, 8, 3, 8), (65, 5, 2, 6), (96, 32, 7, 9), (256, 8, 4, 8), (250, 50, 11, 20), (512, 64, 9, 16),
    (1024, 16, 2, 32), (1000, 8, 8, 22), (63, 63, 3, 3), (128, 64, 40, 32),
]


@pytest.mark.parametrize("E,groups,top,k", CASES)
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("with_bias,best,bf16", [(False, 2, False), (True, 2, True), (False, 1, True), (True, 1, False)])
def test_random_masks(E, groups, top, k, score, with_bias, best, bf16):
    """Every run of every token keeps 0, 1, 2 or more live experts at random."""
    rng = np.random.default_rng([31, E, groups, score, best, with_bias])
    T, size = 41, E // groups
    l = (2 * rng.standard_normal((T, E))).astype(np.float32)
    left = rng.choice(np.array([0, 1, 2, size]), (T, groups, 1))
    order = np.argsort(rng.random((T, groups, size)), 2).argsort(2)
    l = np.where((order < left).reshape(T, E), l, rng.choice(np.array([-np.inf, np.nan], np.float32), (T, E)))
    bias = rng.standard_normal(E).astype(np.float32) if with_bias else None
    print(f"masks E={E} groups={groups}/{top} k={k} score={score} bias={with_bias} best={best}", flush=True)
    check(l, k, bf16, score=score, bias=bias, groups=groups, top_groups=top, group_best=best, renormalize=not with_bias)


@pytest.mark.parametrize("best", [1, 2])
def test_biases_that_are_not_finite_among_masks(best):
    """A live expert with the smallest choice (a bias of minus infinity or NaN) still leads its run past masked ones."""
    rng = np.random.default_rng(32)
    l = rng.standard_normal((30, 48)).astype(np.float32)
    l[rng.random(l.shape) < 0.7] = -np.inf
    bias = rng.choice(np.array([0, 0.5, -np.inf, np.nan, np.inf], np.float32), 48)
    for groups, top, k in ((12, 5, 8), (24, 3, 6), (4, 2, 20)):
        for score in (0, 1):
            check(l, k, score=score, bias=bias, groups=groups, top_groups=top, group_best=best)
