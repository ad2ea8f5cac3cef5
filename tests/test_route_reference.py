"""The router's 64-bit reference on small cases whose answer is written out, and against the older reference where no
expert is masked out."""
import numpy as np
import pytest

import route_reference as RR
import w4_reference as R

INF = np.inf
PAIRS = dict(groups=2, top_groups=1)


@pytest.mark.parametrize("logits,kw,ids,weights", [
    ([-INF, -INF, -INF, 3], PAIRS, [3], [1.0]),                                   # one live expert, behind a masked run
    ([-INF, -INF, 5, -INF], PAIRS, [2], [1.0]),
    ([-INF, -INF, np.nan, 3], dict(PAIRS, score=1), [3], [1.0]),
    ([-INF, -INF, -INF, 3], dict(PAIRS, group_best=1), [3], [1.0]),
    ([-INF, -INF, -INF, 3], dict(PAIRS, bias=[9, 9, 9, -9]), [3], [1.0]),         # masked experts' biases count for nothing
    ([-5, -5, 4, -INF], PAIRS, [2], [1.0]),                                       # 0.9998 alone against two of 0.0001
    ([1, 1, 1.2, -INF], dict(PAIRS, score=1), [0], [1.0]),                        # 0.73 twice against 0.77 alone
    ([-INF] * 4, PAIRS, [0], [0.0]),
    ([-INF, -INF, -INF, -1e30], dict(PAIRS, bias=[0, 0, 0, -INF]), [3], [1.0]),   # live with the smallest choice
    ([-INF, 2, -INF, 3], dict(groups=2, top_groups=2, k=4, renormalize=False, score=1), [3, 1, 0, 2],
     [1 / (1 + np.exp(-3.0)), 1 / (1 + np.exp(-2.0)), 0, 0]),
])
def test_written_out(logits, kw, ids, weights):
    kw = dict(kw)
    got_ids, got_w = RR.route(np.array([logits], np.float32), kw.pop("k", 1), **kw)
    assert got_ids[0].tolist() == ids and np.allclose(got_w[0], weights, rtol=1e-15, atol=0)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("with_bias", [False, True])
def test_agrees_with_the_older_reference_without_masks(score, with_bias):
    rng = np.random.default_rng([1, score, with_bias])
    l = np.round(2 * rng.standard_normal((20, 60)), 1).astype(np.float32)         # many equal logits
    bias = rng.standard_normal(60).astype(np.float32) if with_bias else None
    for groups, top, best in ((1, 1, 2), (5, 2, 2), (5, 2, 1), (60, 7, 2), (30, 4, 2)):
        a = RR.route(l, 5, score, bias, groups, top, best, True, 2.5)
        b = R.route(l, 5, score, bias, groups, top, best, True, 2.5)
        assert np.array_equal(a[0], b[0]) and np.allclose(a[1], b[1], rtol=1e-14, atol=0)
