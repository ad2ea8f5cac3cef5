"""NaN and infinities in rows that are rounded to codes: the scale of the token (group, head) that holds one is NaN, so that
it shows in whatever reads the codes, and every other row has the bits that it has without them."""
import numpy as np
import pytest

import layer_reference as R
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu

BAD = {"nan": 0x7FC0, "-nan": 0xFFC1, "inf": 0x7F80, "-inf": 0xFF80}


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def same(a, b):
    return np.array_equal(host(a).view(np.uint8), host(b).view(np.uint8))


def norm(kind, x, gamma):
    torch, q = torch_mod(), Q()
    M, K = x.shape
    codes = torch.empty((M, K), dtype=torch.int8 if kind == "int8" else torch.uint8, device="cuda")
    s = torch.empty((M, K // 128) if kind == "block" else (M,), device="cuda")
    if kind == "int8":
        q.qlin_norm_int8(dev(x), dev(gamma), codes, s)
    else:
        q.qlin_norm_fp8(dev(x), dev(gamma), codes, s, group=128 if kind == "block" else 0)
    return codes, s


@pytest.mark.parametrize("kind", ["int8", "fp8", "block"])
@pytest.mark.parametrize("K", [128, 512, 2048, 4096, 8192, 32768, 33280])     # every form of the kernel
@pytest.mark.parametrize("bad", BAD)
def test_norm(kind, K, bad):
    rng = np.random.default_rng([1, K])
    x, gamma = R.bits(rng.standard_normal((6, K))), R.bits(1 + 0.2 * rng.standard_normal(K))
    codes, s = norm(kind, x, gamma)
    assert np.isfinite(host(s)).all()
    for row, channel in ((1, 0), (4, K - 1), (5, K // 2 + 3)):
        y = x.copy()
        y[row, channel] = BAD[bad]
        got, t = norm(kind, y, gamma)
        of_bad = host(t)[row, channel // 128] if kind == "block" else host(t)[row]
        assert np.isnan(of_bad), (row, channel)
        others = np.arange(6) != row
        assert same(got[others], codes[others]) and same(t[others], s[others])
    for channel in (0, K - 1):     # a weight of the norm: every row has it
        g = gamma.copy()
        g[channel] = BAD[bad]
        t = host(norm(kind, x, g)[1])
        assert np.isnan(t[:, channel // 128] if kind == "block" else t).all(), channel


def written(kind, k, v, rope, positions, gamma, slots, pages, page):
    torch, q = torch_mod(), Q()
    T, kv_heads, dim = k.shape
    cache = q.KVCache.empty(pages, kv_heads, page, dim, {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[kind])
    more = dict(rope=rope, positions=dev(positions)) if rope else {}
    q.qlin_cache_write(cache, dev(slots), dev(k), dev(v), k_gamma=None if gamma is None else dev(gamma), **more)
    return cache


def read(cache, slots):
    torch, q = torch_mod(), Q()
    k, v = (torch.empty((len(slots), cache.kv_heads, cache.dim), dtype=torch.int16, device="cuda") for _ in range(2))
    q.qlin_cache_read(cache, dev(slots), k, v)
    return R.value(host(k)), R.value(host(v))


def attend(cache, queries, table, lengths):
    torch, q = torch_mod(), Q()
    out = torch.empty(queries.shape, dtype=torch.int16, device="cuda")
    work = torch.empty(q.qlin_attn_decode_workspace(queries.shape[1], cache), dtype=torch.uint8, device="cuda")
    q.qlin_attn_decode(dev(queries), cache, dev(table), dev(lengths), out, work)
    return host(out)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("dim,dims,interleaved", [(16, 0, False), (64, 32, False), (80, 48, True), (128, 128, False), (144, 0, False), (256, 96, True)])
@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("bad", BAD)
def test_cache(kind, dim, dims, interleaved, normed, bad):
    """Token 3 of two sequences of 6 tokens: its key in head 1, its value in head 2."""
    q = Q()
    rng = np.random.default_rng([2, dim])
    T, kv_heads, page, pages = 12, 3, 16, 3
    k, v = (R.bits(rng.standard_normal((T, kv_heads, dim))) for _ in range(2))
    gamma = R.bits(1 + 0.2 * rng.standard_normal(dim)) if normed else None
    rope = q.Rope(dims, interleaved=interleaved) if dims else None
    positions = np.arange(T, dtype=np.int32) % 6
    table = np.array([[2], [0]], np.int32)
    slots = (np.repeat(table[:, 0], 6) * page + positions).astype(np.int32)
    lengths = np.array([6, 6], np.int32)
    queries = R.bits(rng.standard_normal((2, 6, dim)))
    args = rope, positions, gamma, slots, pages, page
    good = written(kind, k, v, *args)
    gk, gv = read(good, slots)
    ga = attend(good, queries, table, lengths)
    assert np.isfinite(gk).all() and np.isfinite(R.value(ga)).all()
    for channel in (0, dim // 2 + 1, dim - 1):
        bk, bv = k.copy(), v.copy()
        bk[3, 1, channel] = bv[3, 2, channel] = BAD[bad]
        cache = written(kind, bk, bv, *args)
        hit = np.zeros((pages, kv_heads, page), bool)
        for n, head in (("k", 1), ("v", 2)):
            hit[:] = False
            hit[2, head, 3] = True
            s, codes = host(getattr(cache, n + "_scale")), host(getattr(cache, n))
            assert np.isnan(s[hit]).all(), n
            assert np.array_equal(s[~hit], host(getattr(good, n + "_scale"))[~hit])
            assert np.array_equal(codes[~hit], host(getattr(good, n))[~hit])
        for got, want, head in zip(read(cache, slots), (gk, gv), (1, 2)):
            assert np.isnan(got[3, head]).all()
            got[3, head] = want[3, head]
            assert np.array_equal(got, want)
        y = attend(cache, queries, table, lengths)
        assert np.isnan(R.value(y[0, 2:])).all(), "heads 2 to 5 read kv heads 1 and 2"
        y[0, 2:] = ga[0, 2:]
        assert np.array_equal(y, ga)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_unrounded_cache(dim):
    rng = np.random.default_rng([3, dim])
    k, v = (R.bits(rng.standard_normal((6, 2, dim))) for _ in range(2))
    slots, lengths, table = np.arange(6, dtype=np.int32), np.array([6], np.int32), np.array([[0]], np.int32)
    queries = R.bits(rng.standard_normal((1, 4, dim)))
    good = attend(written("bf16", k, v, None, None, None, slots, 1, 16), queries, table, lengths)
    k[2, 0, 5] = v[4, 1, 7] = BAD["nan"]
    cache = written("bf16", k, v, None, None, None, slots, 1, 16)
    gk, gv = read(cache, slots)
    assert np.isnan(gk[2, 0, 5]) and np.isnan(gv[4, 1, 7]) and np.isnan(gk).sum() == np.isnan(gv).sum() == 1
    y = attend(cache, queries, table, lengths)
    assert np.isnan(R.value(y[0, :2])).all() and np.isnan(R.value(y[0, 2:, 7])).all()
    y[0, :2], y[0, 2:, 7] = good[0, :2], good[0, 2:, 7]
    assert np.array_equal(y, good)
