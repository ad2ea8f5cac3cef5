"""Attention of one new token over the paged cache against the definition in 64 bits, at the lengths, pages, windows and
head layouts where it can go wrong."""
import numpy as np
import pytest

import layer_reference as R
import oracle as O
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


class Case:
    """A batch: the cache's contents, tables in random order, queries."""

    def __init__(self, seed, kind, lengths, heads, kv_heads, dim, page, spare=2, columns=None, sharp=1.5):
        torch, q = torch_mod(), Q()
        rng = self.rng = np.random.default_rng([seed, heads, dim, page, len(lengths)])
        self.kind, self.page, self.heads = kind, page, heads
        self.lengths = np.array(lengths, np.int32)
        held = [-(-max(0, n) // page) for n in lengths]
        self.columns = max([1] + held) if columns is None else columns
        self.pages = sum(held) + spare
        order = rng.permutation(self.pages).astype(np.int32)
        self.table = rng.integers(-3, self.pages + 3, (len(lengths), self.columns)).astype(np.int32)   # behind a length: anything
        first = 0
        for i, n in enumerate(held):
            self.table[i, :n] = order[first:first + n][:self.columns]
            first += n
        shape = (self.pages, kv_heads, page, dim)
        self.cache = q.KVCache.empty(*shape, {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[kind])
        self.raw, self.scales = {}, {}
        for n in ("k", "v"):
            x = rng.standard_normal(shape) + (0.3 if n == "v" else 0.0)
            if kind == "bf16":
                self.raw[n] = R.bits(x)
            elif kind == "int8":
                self.raw[n] = np.clip(np.rint(x * 32), -127, 127).astype(np.int8)
            else:
                self.raw[n] = O.e4m3_encode(np.clip(x * 64, -448, 448).astype(np.float32)).astype(np.uint8)
            self.scales[n] = None if kind == "bf16" else (rng.uniform(0.5, 1.5, shape[:3]) / (32 if kind == "int8" else 64)).astype(np.float32)
        self.q = R.bits(rng.standard_normal((len(lengths), heads, dim)) * sharp)

    def values(self, n):
        raw = self.raw[n]
        v = R.value(raw) if self.kind == "bf16" else raw.astype(np.float64) if self.kind == "int8" else O.e4m3_decode(raw)
        return v if self.scales[n] is None else v * self.scales[n].astype(np.float64)[..., None]

    def load(self):
        torch = torch_mod()
        for n in ("k", "v"):
            t = getattr(self.cache, n)
            (t.view(torch.int16) if self.kind == "bf16" else t).copy_(dev(self.raw[n]))
            if self.scales[n] is not None:
                getattr(self.cache, n + "_scale").copy_(dev(self.scales[n]))
        return self

    def run(self, window=0, scale=None, stream=None):
        torch, q = torch_mod(), Q()
        need = q.qlin_attn_decode_workspace(self.heads, self.cache)
        work = torch.full((need + 64,), 0xEE, dtype=torch.uint8, device="cuda")
        raw = torch.full((self.q.size + 32,), 0x1234, dtype=torch.int16, device="cuda")
        out = raw[:-32].view(self.q.shape)
        q.qlin_attn_decode(dev(self.q), self.cache, dev(self.table), dev(self.lengths), out, work[:need], scale=scale, window=window,
                           stream=stream)
        torch.cuda.synchronize()
        assert int((raw[-32:] != 0x1234).sum()) == 0 and int((work[need:] != 0xEE).sum()) == 0, "written past a buffer"
        return host(out)

    def check(self, got, window=0, scale=None):
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        scale = float(np.float32(scale))
        with np.errstate(invalid="ignore"):
            ref, room = R.attention(R.value(self.q), self.values("k"), self.values("v"), self.table, self.lengths, self.page, window, scale)
        stay = np.isnan(ref) & (self.lengths < 0)[:, None, None]
        assert (got[stay] == 0x1234).all(), "rows without a sequence were written"
        y = R.value(got)[~stay]
        off = np.abs(y - ref[~stay]) - (np.abs(ref[~stay]) * R.HALF + room[~stay] * (1 + R.HALF))
        assert (off <= 1e-30).all(), float(off.max())


KINDS = ["bf16", "int8", "fp8"]
EDGES = [0, -1, 1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 255, 257, 400]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [16, 48, 64])
def test_lengths_at_the_edges(kind, page):
    c = Case(1, kind, EDGES, 8, 2, 128, page).load()
    c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 16), (2, 2, 32), (3, 1, 64), (20, 4, 64), (8, 8, 80), (5, 1, 96), (16, 1, 128), (17, 1, 128),
                                                (40, 1, 64), (33, 3, 48), (32, 8, 128), (4, 2, 144), (6, 2, 192), (8, 1, 256), (34, 2, 256),
                                                (7, 7, 112)])
@pytest.mark.parametrize("columns", [None, 300])    # one launch, or items that are joined
def test_head_layouts(kind, heads, kv_heads, dim, columns):
    c = Case(2, kind, [130, 7, 0, 33, 64, 290], heads, kv_heads, dim, 32, columns=columns).load()
    c.check(c.run())
    c.check(c.run(window=50), window=50)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths", [[1], [777], [5000], [9000, 3, 0, 0, 12, 2500], [100] * 70, [0] * 65 + [300] + [0] * 70 + [40], [0], [-1, -7],
                                     [0, 0, 0]])
@pytest.mark.parametrize("columns", [None, 700])
def test_split_and_joined(kind, lengths, columns):
    c = Case(3, kind, lengths, 4, 2, 64, 16, columns=columns).load()
    c.check(c.run())


@pytest.mark.parametrize("S", [1023, 1024, 1025, 3000])
def test_many_sequences(S):
    rng = np.random.default_rng(S)
    lengths = rng.integers(-1, 20, S)
    lengths[[0, S // 2, S - 1]] = [700, 1300, 333]
    c = Case(14, "int8", lengths.tolist(), 2, 1, 32, 16, columns=200).load()
    c.check(c.run())


def test_one_group_of_heads_and_many_parts():
    """A single kv head: up to a thousand partial sums of one sequence, the join's loops over 64 and over 16 of them."""
    for dim, n in ((64, 70000), (128, 9000), (256, 40000)):
        c = Case(15, "fp8", [n, 100, 0], 17, 1, dim, 64).load()
        c.check(c.run())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window", [1, 5, 16, 31, 33, 100, 4096, 1 << 40])
def test_windows(kind, window):
    c = Case(4, kind, [0, 1, 16, 33, 100, 259, 1800], 6, 2, 128, 48).load()
    # pages wholly before a window are given back: their entries may name anything
    for s, n in enumerate(c.lengths):
        gone = max(0, int(n) - window) // c.page
        c.table[s, :gone] = [(-9, c.pages + 100, 0)[i % 3] for i in range(gone)]
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_masked_places_hold_anything(kind):
    """NaN and infinities behind the length, before the window and in every page of nobody."""
    c = Case(5, kind, [19, 33, 100, 16, 250], 4, 2, 64, 32)
    live = np.zeros((c.pages, c.page), bool)
    window = 70
    for s, n in enumerate(c.lengths):
        t = np.arange(max(0, n - window), n)
        live[c.table[s][t // c.page], t % c.page] = True
    dead = ~live
    for n in ("k", "v"):
        raw = c.raw[n].swapaxes(1, 2)
        raw[dead] = {"bf16": 0x7FC0, "int8": -128, "fp8": 0x7F}[c.kind]
        if c.kind == "bf16":
            raw[dead & (np.arange(c.page) % 2 == 0)[None]] = 0xFF80
        if c.scales[n] is not None:
            s = c.scales[n].swapaxes(1, 2)
            s[dead] = np.nan
            s[dead & (np.arange(c.page) % 3 == 0)[None]] = np.inf
    c.load()
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_pages_outside_the_cache_are_left_out(kind):
    c = Case(6, kind, [200, 90, 64, 500], 4, 1, 128, 32).load()
    c.table[0, 2] = -1
    c.table[1, 0] = c.pages
    c.table[2, :] = 2147483647                  # nothing is left: zero
    c.table[3, ::2] = -2147483648
    got = c.run()
    assert (got[2] == 0).all()
    c.check(got)


def test_lengths_past_the_table():
    c = Case(7, "fp8", [500, 40, 3], 4, 2, 64, 16, columns=5).load()
    assert c.columns * c.page == 80
    c.check(c.run())
    c.lengths[:] = 2147483647
    c.table[:] = np.clip(c.table, 0, c.pages - 1)
    c.check(c.run())


def test_sharp_softmax_and_scales():
    """Scores far apart, in either order; scales of other heads; a scale of zero and a negative one."""
    for scale in (None, 1.0, 0.0, -0.3):
        c = Case(8, "int8", [700, 33, 5], 8, 2, 128, 16, sharp=6.0).load()
        c.check(c.run(scale=scale), scale=scale)
    c = Case(9, "fp8", [300], 2, 1, 64, 16)
    c.scales["v"][:] = np.where(np.arange(16) % 2, 1e-30, 1e30).astype(np.float32)[None, None]
    c.scales["k"][:, :, 3] = 0
    c.load()
    c.check(c.run())


def test_pages_shared_by_sequences():
    c = Case(10, "int8", [96, 96, 96, 64], 8, 4, 64, 32).load()
    c.table[1:, :2] = c.table[0, :2]            # a prefix that all of them have
    c.check(c.run())


def test_a_long_sequence_and_a_cache_past_4_gib():
    torch, q = torch_mod(), Q()
    pages, kv_heads, page, dim = 66000, 4, 128, 128          # 4.3 GB of keys
    cache = q.KVCache.empty(pages, kv_heads, page, dim, torch.int8)
    rng = np.random.default_rng(12)
    n = 3000
    used = np.array([pages - 1 - 7 * i for i in range(-(-n // page))], np.int32)
    k, v = (np.clip(np.rint(rng.standard_normal((len(used), kv_heads, page, dim)) * 32), -127, 127).astype(np.int8) for _ in range(2))
    at = torch.from_numpy(used.astype(np.int64)).cuda()
    cache.k[at], cache.v[at] = dev(k), dev(v)
    cache.k_scale[at], cache.v_scale[at] = 1 / 32, 1 / 16
    qb = R.bits(rng.standard_normal((1, 8, dim)))
    out = torch.empty((1, 8, dim), dtype=torch.int16, device="cuda")
    work = torch.empty(q.qlin_attn_decode_workspace(8, cache), dtype=torch.uint8, device="cuda")
    q.qlin_attn_decode(dev(qb), cache, dev(used[None]), dev(np.array([n], np.int32)), out, work)
    scale = float(np.float32(dim ** -0.5))
    ref, room = R.attention(R.value(qb), k / 32.0, v / 16.0, np.arange(len(used))[None], [n], page, 0, scale)
    assert (np.abs(R.value(host(out)) - ref) <= np.abs(ref) * R.HALF + room * (1 + R.HALF)).all()


def test_the_same_call_gives_the_same_bits():
    c = Case(13, "fp8", [5000, 77, 1200], 8, 2, 128, 64).load()
    first = c.run()
    for _ in range(4):
        assert np.array_equal(first, c.run())
