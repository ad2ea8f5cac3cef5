"""Routing to experts against the definition in 64 bits: the chosen experts are equal, the weights within the
rounding to f32 of a value evaluated in f64 (a relative 2^-24; 2^-23 leaves room for the f64 steps)."""
import numpy as np
import pytest

import w4_reference as R
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def run(logits, k, bf16=False, **kw):
    """-> ids, weights; logits f32 array, sent as bf16 where asked."""
    torch = torch_mod()
    T = logits.shape[0]
    l = torch.from_numpy(np.ascontiguousarray(logits, np.float32)).cuda()
    if bf16:
        l = l.to(torch.bfloat16)
    bias = kw.pop("bias", None)
    ids = torch.full((T * k + 16,), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T * k + 16,), 7.0, device="cuda")
    Q().qlin_route(l, ids[:T * k].view(T, k), w[:T * k].view(T, k), bias=None if bias is None else dev(bias), **kw)
    assert (host(ids)[T * k:] == -7).all() and (host(w)[T * k:] == 7.0).all(), "written past the outputs"
    return host(ids)[:T * k].reshape(T, k), host(w)[:T * k].reshape(T, k)


def check(logits, k, bf16=False, score=0, bias=None, groups=1, top_groups=1, group_best=2, renormalize=True, scale=1.0):
    ids, w = run(logits, k, bf16, score=score, bias=bias, groups=groups, top_groups=top_groups, group_best=group_best,
                 renormalize=renormalize, scale=scale)
    if bf16:
        logits = R.bf16_values(R.bf16_bits(logits)).astype(np.float32).reshape(logits.shape)
    rid, rw = R.route(logits, k, score, bias, groups, top_groups, group_best, renormalize, scale)
    assert np.array_equal(ids, rid)
    assert (np.abs(w - rw) <= 2.0 ** -23 * np.abs(rw) + 2.0 ** -149).all()   # the last term: f32's smallest step


CASES = [  # T, E, k, groups, top_groups
    (1, 1, 1, 1, 1), (1, 128, 8, 1, 1), (3, 2, 2, 1, 1), (333, 60, 4, 1, 1), (5, 64, 32, 1, 1), (7, 65, 6, 5, 2), (9, 100, 1, 4, 4),
    (130, 256, 8, 8, 4), (64, 250, 10, 5, 3), (17, 512, 16, 64, 9), (33, 1024, 32, 16, 1), (21, 1000, 22, 8, 8), (40, 63, 3, 63, 3),
]


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("T,E,k,groups,top", CASES)
@pytest.mark.parametrize("with_bias,best,bf16", [(False, 2, False), (True, 2, False), (False, 1, True), (True, 1, True)])
def test_against_the_definition(T, E, k, groups, top, score, with_bias, best, bf16):
    rng = np.random.default_rng([T, E, k, score, best])
    logits = (2 * rng.standard_normal((T, E))).astype(np.float32)     # bf16: many equal logits
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    print(f"route T={T} E={E} k={k} groups={groups}/{top} score={score} bias={with_bias} best={best}", flush=True)
    check(logits, k, bf16, score, bias, groups, top, best, renormalize=best == 2, scale=2.5 if with_bias else 1.0)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(score, with_bias):
    """-infinity and NaN mask experts out: fewer left than choices, whole groups, a whole row; +infinity leads."""
    rng = np.random.default_rng(11)
    l = rng.standard_normal((8, 96)).astype(np.float32)
    l[0, 5:] = -np.inf                     # five experts left
    l[1, :] = -np.inf                      # none left
    l[2, ::2] = np.nan
    l[3, 12:24] = -np.inf                  # a whole group
    l[4, [3, 50]] = np.inf
    l[5, :] = np.finfo(np.float32).min     # the type's lowest value is a logit like any other
    l[6, :90] = np.finfo(np.float32).min
    bias = rng.standard_normal(96).astype(np.float32) if with_bias else None
    check(l, 8, score=score, bias=bias)
    check(l, 8, score=score, bias=bias, groups=8, top_groups=3)
    check(l, 8, score=score, bias=bias, renormalize=False, scale=3.0)
    ids, w = run(l, 8, score=score, bias=bias)
    assert (w[1] == 0).all()
    assert (w[0][ids[0] >= 5] == 0).all()


def test_equal_choices_take_the_lowest_index():
    l = np.zeros((4, 200), np.float32)
    l[1, 100:] = 1.0
    l[2, [199, 7, 64]] = 2.0
    for kw in ({}, {"bias": np.zeros(200, np.float32)}, {"groups": 4, "top_groups": 2}, {"score": 1}):
        check(l, 6, **kw)
    assert run(l, 6)[0][2].tolist() == [7, 64, 199, 0, 1, 2]


def test_biases_that_are_not_finite():
    rng = np.random.default_rng(12)
    l = rng.standard_normal((6, 40)).astype(np.float32)
    bias = np.zeros(40, np.float32)
    bias[[1, 2, 3, 30]] = [np.inf, -np.inf, np.nan, np.inf]
    check(l, 5, score=1, bias=bias)
    check(l, 40 // 2, score=0, bias=bias, groups=2, top_groups=2)
    l[:, [3, 7, 8]] = -np.inf              # masked experts come after one with the smallest bias
    check(l, 32, score=1, bias=np.where(np.arange(40) > 20, -np.inf, bias).astype(np.float32)[:40], groups=1)


def test_neighbouring_scores_are_told_apart():
    """Logits one f32 step apart: the choice is the exact order, with a bias as without."""
    base = np.full(128, 0.3, np.float32)
    for i in range(1, 128):
        base[i] = np.nextafter(base[i - 1], np.float32(1), dtype=np.float32)
    rng = np.random.default_rng(13)
    l = np.stack([rng.permutation(base) for _ in range(16)])
    for score in (0, 1):
        check(l, 8, score=score)
        check(l, 8, score=score, bias=np.full(128, 0.25, np.float32))


def test_many_tokens():
    rng = np.random.default_rng(14)
    l = rng.standard_normal((3001, 32)).astype(np.float32)
    check(l, 2, score=1, bias=(0.1 * rng.standard_normal(32)).astype(np.float32), groups=4, top_groups=2, scale=2.5)
