"""The exact inputs are what their users take them for: sums that f32 holds, gates past 20, and results that a rounding
of h to one bf16 changes."""
import numpy as np
import pytest

import w4_exact as X
import w4_reference as R


def fits_f32(x, w, unit):
    """Every partial sum of products of inputs and codes or zero points, in steps of `unit`, stays below 2^24 steps."""
    codes, scales, zp = w
    most = max(15, 0 if zp is None else int(zp.max()))
    top = R.bf16_values(scales).max()
    low = R.bf16_values(scales).min()
    assert (x / unit == np.round(x / unit)).all()
    return np.abs(x).sum(1).max() / unit * most * top / min(low, 1.0) < 2 ** 24


@pytest.mark.parametrize("M,I,K,group,zeros", X.SWIGLU)
def test_swiglu_inputs(M, I, K, group, zeros):
    x, gate, up = X.swiglu_case(1, M, I, K, group, zeros)
    assert np.array_equal(R.bf16_values(R.bf16_bits(x)).reshape(x.shape), x)
    _, g = X.swiglu(x, gate, up)
    assert g.min() >= 20 and np.float32(1) + np.exp(np.float32(-20)) == 1
    assert fits_f32(x, gate, 1) and fits_f32(x, up, 1)


@pytest.mark.parametrize("case,low", [(c, True) for c in X.LOW] + [(c, False) for c in X.ANY])
def test_experts_inputs(case, low):
    x, ids, wt, ws = X.experts_case(2, *case, low)
    assert np.array_equal(R.bf16_values(R.bf16_bits(x)).reshape(x.shape), x)
    one = lambda w, e: tuple(None if t is None else t[e] for t in w)  # noqa: E731
    for e in (0, int(ids.max())):
        g, u = (x @ R.dequantize(one(w, e))[0].T for w in ws[:2])
        assert np.isin(g, [64, 128]).all() and u.min() >= 256 and u.max() <= 505
        assert fits_f32(x, one(ws[0], e), 1) and fits_f32(x, one(ws[1], e), 1) and fits_f32(g * u, one(ws[2], e), 64)
    exact = X.experts(x, ids, wt, ws, 2)
    # sums over groups and slots, in any order: steps of 64 / 4 (scales and weights down to 1/2), 2^24 of them at most
    assert (exact % 16 == 0).all() and X.experts(x, ids, wt, ws, 2, magnitudes=True).max() < 16 * 2 ** 24
    assert np.array_equal(exact, R.experts(x, ids, wt, *ws, case[5])[0])   # two parts lose nothing
    once = X.experts(x, ids, wt, ws, 1)
    if low:
        assert (once == 0).all() and (exact != 0).mean() > 0.9        # one part loses all
    else:
        assert np.array_equal(once, exact)


def test_a_rounding_of_h_shows():
    """Planted in the oracle: one bf16 of h, and a low part of half its value, are both told from the right result."""
    for case in X.LOW:
        x, ids, wt, ws = X.experts_case(2, *case, True)
        right = R.bf16_bits(X.experts(x, ids, wt, ws, 2))
        assert (R.bf16_bits(X.experts(x, ids, wt, ws, 1)) != right).mean() > 0.9
        assert (R.bf16_bits(X.experts(x, ids, wt, ws, 2) / 2) != right).mean() > 0.9
