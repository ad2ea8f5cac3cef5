"""Every form of the attention against the definition in 64 bits."""
import numpy as np
import pytest

import layer_forms as F
import layer_reference as R
import test_attn_gpu as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", F.KINDS)
@pytest.mark.parametrize("case", F.ATTENTION, ids=lambda c: "-".join(map(str, (len(c[0]),) + c[1:])))
def test_attention(case, kind):
    lengths, heads, kv_heads, dim, page, columns, window = case
    c = A.Case(21, kind, lengths, heads, kv_heads, dim, page, columns=columns).load()
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("kind", F.KINDS)
@pytest.mark.parametrize("dim", [64, 128, 144, 256])
@pytest.mark.parametrize("columns", [16, 40])     # one launch, or items that are joined
def test_masked_places_hold_anything(kind, dim, columns):
    """NaN and infinities behind the length, before the window and in the pages of nobody; pages outside the cache."""
    c = A.Case(22, kind, [19, 33, 100, 16, 250, 256], 8, 2, dim, 16, columns=columns)
    window = 70
    c.table[4, 12] = -1
    c.table[5, 13:] = [c.pages, 2147483647, -2147483648] + [7] * (columns - 16)
    live = np.zeros((c.pages, c.page), bool)
    for s, n in enumerate(c.lengths):
        t = np.arange(max(0, n - window), n)
        p = c.table[s][t // c.page]
        ok = (p >= 0) & (p < c.pages)
        live[p[ok], t[ok] % c.page] = True
    dead = ~live
    for n in ("k", "v"):
        raw = c.raw[n].swapaxes(1, 2)
        raw[dead] = {"bf16": 0x7FC0, "int8": -128, "fp8": 0x7F}[kind]
        if kind == "bf16":
            raw[dead & (np.arange(c.page) % 2 == 0)[None]] = 0xFF80
        else:
            s = c.scales[n].swapaxes(1, 2)
            s[dead] = np.nan
            s[dead & (np.arange(c.page) % 3 == 0)[None]] = np.inf
    c.load()
    c.check(c.run(window=window), window=window)


@pytest.mark.parametrize("kind", ["int8", "fp8"])
@pytest.mark.parametrize("exponent", [-110, -117, -120, -123, -126])
def test_small_value_scales(kind, exponent):
    """Scales of values near the end of the f32 range: a product p * v_scale is off by 2^-134 at most besides its relative
    error (half a step of a subnormal bf16), times a code, over the tokens; the sums and the output, half a step of their
    subnormals (2^-150 and 2^-134)."""
    c = A.Case(23, kind, [300, 33], 4, 2, 64, 16)
    scales = np.ldexp(c.scales["v"].astype(np.float64) * 32, exponent)
    c.scales["v"] = scales.astype(np.float32)
    y = R.value(c.load().run())
    ref, room = R.attention(R.value(c.q), c.values("k"), c.values("v"), c.table, c.lengths, c.page, 0, float(np.float32(64 ** -0.5)))
    tokens = np.array(c.lengths)[:, None, None]
    room = room + tokens * (2.0 ** -134 * R.MOST[kind] + 4 * 2.0 ** -150) + 2.0 ** -134
    assert (np.abs(y - ref) <= np.abs(ref) * R.HALF + room * (1 + R.HALF)).all()
