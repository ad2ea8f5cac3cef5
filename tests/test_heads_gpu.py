"""Rotary positions, the cache's write and its read against their definitions in 64 bits."""
import numpy as np
import pytest

import layer_reference as R
import oracle as O
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def draw(rng, *shape):
    return R.bits(rng.standard_normal(shape) * np.where(np.arange(shape[-1]) % 23 == 3, 6.0, 1.0))


def gammas(rng, dim, on):
    return [R.bits(1 + 0.3 * rng.standard_normal(dim)) if on else None for _ in range(2)]


def some_positions(rng, T):
    p = rng.integers(0, 131072, T).astype(np.int32)
    p[:4] = np.array([0, 1, 2147483647, -5], np.int32)[:T]
    return p


def device(a):
    return None if a is None else dev(a)


def within(y, ref, slack, what=""):
    off = np.abs(y - ref) - (np.abs(ref) * R.HALF + slack * (1 + R.HALF))
    assert (off <= 1e-30).all(), (what, float(off.max()))


ROPE = [  # T, heads, dim, dims, interleaved, norm
    (1, 1, 16, 16, False, False), (3, 2, 32, 16, True, True), (5, 3, 64, 64, False, False), (6, 13, 64, 32, True, False),
    (7, 1, 80, 80, False, True), (9, 5, 80, 48, True, True), (5, 7, 96, 16, False, False), (4, 32, 128, 128, False, True),
    (3, 40, 128, 64, False, False), (11, 33, 128, 112, True, True), (2, 9, 144, 144, False, True), (3, 17, 256, 256, True, False),
    (2, 3, 256, 96, False, True), (70, 4, 128, 128, False, False),
    (1030, 1, 128, 64, False, True), (2050, 2, 64, 64, True, False), (16390, 1, 48, 32, False, False), (1025, 3, 256, 256, False, False),   # several tokens to a workgroup
]


@pytest.mark.parametrize("T,heads,dim,dims,interleaved,norm", ROPE)
@pytest.mark.parametrize("layout", ["own", "in place", "part of a row"])
def test_rope(T, heads, dim, dims, interleaved, norm, layout):
    torch, q = torch_mod(), Q()
    rng = np.random.default_rng([5, T, heads, dim, dims])
    xb, pos, gamma = draw(rng, T, heads, dim), some_positions(rng, T), gammas(rng, dim, norm)[0]
    rope = q.Rope(dims, 5e5, "bands", 8.0, 8192, interleaved=interleaved, strength=1.25 if heads % 2 else None)
    freq = rope.frequencies.cpu().numpy()
    if layout == "part of a row":
        wide = torch.full((T, heads + 3, dim), 0x7FC0, dtype=torch.int16, device="cuda")     # NaN around them
        x = wide[:, 2:2 + heads]
        x.copy_(dev(xb))
        out = torch.full((T, heads + 1, dim), 0x1234, dtype=torch.int16, device="cuda")
        y = out[:, :heads]
    else:
        x = dev(xb)
        y = x if layout == "in place" else torch.full_like(x, 0x1234)
    q.qlin_rope(x, dev(pos), rope, y, gamma=device(gamma), eps=1e-5)
    ref, slack = R.rotate(R.value(xb), pos, freq, dims, interleaved, rope.strength, None if gamma is None else R.value(gamma), 1e-5)
    got = R.value(host(y.contiguous()))
    within(got, ref, slack)
    if not norm:
        assert np.array_equal(host(y.contiguous()).view(np.uint16)[..., dims:], xb[..., dims:]), "channels that do not turn"
    if layout == "part of a row":
        assert int((out[:, heads:] != 0x1234).sum()) == 0 and int((wide[:, :2] != 0x7FC0).sum()) == 0


KINDS = ["bf16", "int8", "fp8"]
WRITE = [  # T, heads, kv_heads, dim, page, dims (0: no rotation), interleaved, norm
    (1, 4, 1, 128, 16, 128, False, False), (5, 0, 2, 64, 48, 0, False, False), (9, 3, 3, 16, 16, 16, True, True),
    (33, 32, 8, 128, 64, 128, False, True), (6, 10, 5, 80, 32, 48, False, False), (4, 8, 2, 256, 16, 256, True, True),
    (7, 0, 4, 96, 16, 96, False, True), (12, 6, 6, 144, 80, 64, True, False), (3, 64, 8, 128, 16, 0, False, True),
    (2, 200, 100, 64, 16, 64, False, False), (1027, 2, 1, 64, 16, 64, False, True), (4099, 0, 1, 64, 48, 0, False, False),
]


def empty_cache(torch, q, kind, pages, kv_heads, page, dim, fill=0x5A):
    dtype = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[kind]
    cache = q.KVCache.empty(pages, kv_heads, page, dim, dtype)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.view(torch.uint8).fill_(fill)
    return cache


def contents(cache, kind, n):
    """-> (values of the codes, raw bytes, scales) of k or v, [pages, page, kv_heads, ...]"""
    torch = torch_mod()
    t = getattr(cache, n)
    raw = host(t.view(torch.int16) if kind == "bf16" else t)
    v = R.value(raw) if kind == "bf16" else raw.astype(np.float64) if kind == "int8" else O.e4m3_decode(raw)
    s = None if kind == "bf16" else host(getattr(cache, n + "_scale"))
    return v.swapaxes(1, 2), raw.swapaxes(1, 2), None if s is None else s.swapaxes(1, 2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,heads,kv_heads,dim,page,dims,interleaved,norm", WRITE)
def test_cache_write(kind, T, heads, kv_heads, dim, page, dims, interleaved, norm):
    torch, q = torch_mod(), Q()
    rng = np.random.default_rng([7, T, heads, kv_heads, dim])
    pages = T // page + 2
    total = pages * page
    wide = draw(rng, T, heads + 2 * kv_heads, dim)
    qb, kb, vb = wide[:, :heads], wide[:, heads:heads + kv_heads], wide[:, heads + kv_heads:]
    pos = some_positions(rng, T)
    slots = rng.permutation(total)[:T].astype(np.int32)
    if T > 4:
        slots[[1, 2, 4]] = [-1, total, -2147483648]
    qg, kg = gammas(rng, dim, norm)
    rope = q.Rope(dims, 1e4, interleaved=interleaved) if dims else None
    cache = empty_cache(torch, q, kind, pages, kv_heads, page, dim)
    qkv = dev(wide)
    qs, ks, vs = qkv.split((heads, kv_heads, kv_heads), 1)
    out = torch.full((T, max(heads, 1), dim), 0x1234, dtype=torch.int16, device="cuda")
    more = dict(q=qs, q_out=out, q_gamma=device(qg)) if heads else {}
    if dims:
        more.update(rope=rope, positions=dev(pos))
    q.qlin_cache_write(cache, dev(slots), ks, vs, k_gamma=device(kg), eps=1e-5, **more)
    assert torch.equal(qkv, dev(wide)), "the inputs changed"

    def turned(b, g):
        if dims:
            return R.rotate(R.value(b), pos, rope.frequencies.cpu().numpy(), dims, interleaved, 1.0, None if g is None else R.value(g), 1e-5)
        x = R.value(b)
        if g is None:
            return x, np.zeros_like(x)
        x = x * R.value(g) / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        return x, np.abs(x) * R.U32 * 60

    if heads:
        within(R.value(host(out)), *turned(qb, qg), "queries")
    live = (slots >= 0) & (slots < total)
    at = (slots[live] // page, slots[live] % page)
    for n, (ref, slack) in (("k", turned(kb, kg)), ("v", (R.value(vb), np.zeros(vb.shape)))):
        values, raw, s = contents(cache, kind, n)
        ref, slack = ref[live], slack[live]
        if kind == "bf16":
            within(values[at], ref, slack, n)
        else:
            Qm = R.MOST[kind]
            a = np.abs(ref).max(-1)
            top = slack.max(-1)
            assert (np.abs(s[at] - a / Qm) <= top / Qm + a / Qm * 4 * R.U32).all(), n + " scales"
            if not slack.any():   # every step is one IEEE operation
                want, scale = R.codes(ref, kind)
                assert np.array_equal(values[at], want) and np.array_equal(s[at], scale)
            x = ref / (a / Qm)[..., None]            # what is rounded, off by the slack and the scale's own
            room = (slack + np.abs(ref) * (top / a)[..., None]) * (Qm / a)[..., None] + np.abs(x) * 4 * R.U32
            step = np.full(x.shape, 0.5) if kind == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10)
            assert (np.abs(values[at] - x) <= step * (1 + 2.0 ** -3 * (kind == "fp8") * (room > 0)) + room).all(), n
        touched = np.zeros(raw.shape[:2], bool)
        touched[at] = True
        untouched = raw[~touched]
        assert (untouched.view(np.uint8) == 0x5A).all(), "places of no slot were written"
        if s is not None:
            assert (s[~touched].view(np.uint8) == 0x5A).all()


def test_cache_write_rows_of_zeros_and_extremes():
    torch, q = torch_mod(), Q()
    kb = np.zeros((4, 2, 64), np.uint16)
    rng = np.random.default_rng(3)
    kb[1] = R.bits(rng.standard_normal((2, 64)) * 2.0 ** -80)
    kb[2] = R.bits(rng.standard_normal((2, 64)) * 2.0 ** 50)
    kb[3, :, 5] = 0xC000                       # -2 alone
    for kind in ("int8", "fp8"):
        cache = empty_cache(torch, q, kind, 1, 2, 16, 64)
        q.qlin_cache_write(cache, dev(np.arange(4, dtype=np.int32)), dev(kb), dev(kb))
        for n in ("k", "v"):
            values, _, s = contents(cache, kind, n)
            want, scale = R.codes(R.value(kb), kind)
            assert np.array_equal(values[0, :4], want) and np.array_equal(s[0, :4], scale)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,kv_heads,dim,page,pages", [(1, 1, 16, 16, 1), (5, 3, 64, 48, 2), (70, 8, 128, 16, 9), (517, 5, 80, 48, 12),
                                                        (33, 2, 256, 64, 2), (9, 40, 256, 16, 3), (300, 1, 96, 32, 11)])
def test_cache_read(kind, n, kv_heads, dim, page, pages):
    torch, q = torch_mod(), Q()
    rng = np.random.default_rng([9, n, dim])
    cache = empty_cache(torch, q, kind, pages, kv_heads, page, dim)
    for m in ("k", "v"):
        shape = (pages, kv_heads, page, dim)
        raw = draw(rng, *shape) if kind == "bf16" else rng.integers(-127, 128, shape).astype(np.int8) if kind == "int8" else \
            (rng.integers(0, 0x7F, shape) | (rng.integers(0, 2, shape) << 7)).astype(np.uint8)
        t = getattr(cache, m)
        (t.view(torch.int16) if kind == "bf16" else t).copy_(dev(raw))
        if kind != "bf16":
            getattr(cache, m + "_scale").copy_(dev(rng.uniform(1e-4, 2, shape[:3]).astype(np.float32)))
    slots = rng.integers(0, pages * page, n).astype(np.int32)       # some twice
    if n > 4:
        slots[[1, 3]] = [-1, pages * page]
    raws = [torch.full((n * kv_heads * dim + 32,), 0x1234, dtype=torch.int16, device="cuda") for _ in range(2)]
    k, v = (r[:-32].view(n, kv_heads, dim) for r in raws)
    q.qlin_cache_read(cache, dev(slots), k, v)
    live = (slots >= 0) & (slots < pages * page)
    for m, got, raw in (("k", k, raws[0]), ("v", v, raws[1])):
        values, _, s = contents(cache, kind, m)
        at = (slots[live] // page, slots[live] % page)
        want = values[at] if s is None else (values[at].astype(np.float32) * s[at][..., None]).astype(np.float32)
        assert np.array_equal(host(got).view(np.uint16)[live], R.bits(want)), m
        assert (host(got)[~live] == 0x1234).all() and int((raw[-32:] != 0x1234).sum()) == 0


def test_cache_past_4_gib():
    """Slots at the end of a cache of more than 2^32 bytes: written and read back."""
    torch, q = torch_mod(), Q()
    pages, kv_heads, page, dim = 40000, 8, 128, 128                 # 5.2 GB of keys
    cache = q.KVCache.empty(pages, kv_heads, page, dim, torch.int8)
    rng = np.random.default_rng(4)
    slots = np.array([pages * page - 1, 0, pages * page - 129, 33000 * 128 + 7], np.int32)
    kb, vb = draw(rng, 4, kv_heads, dim), draw(rng, 4, kv_heads, dim)
    q.qlin_cache_write(cache, dev(slots), dev(kb), dev(vb))
    k, v = (torch.empty((4, kv_heads, dim), dtype=torch.int16, device="cuda") for _ in range(2))
    q.qlin_cache_read(cache, dev(slots), k, v)
    for got, b in ((k, kb), (v, vb)):
        want, s = R.codes(R.value(b), "int8")
        assert np.array_equal(host(got).view(np.uint16), R.bits((want.astype(np.float32) * s[..., None]).astype(np.float32)))
    assert int(cache.k_scale.count_nonzero()) == 4 * kv_heads
