"""The most rows, tokens and sequences that the norm, rotary, cache and attention calls take: several launches' worth, of
which the first, the last and those at the borders are compared with calls of their own."""
import pytest

from gpu_helpers import torch_mod

pytestmark = pytest.mark.gpu
MOST = 1 << 24


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def rows(torch):
    at = [0, 1, 7, (1 << 21) - 1, 1 << 21, (1 << 23) - 1, 1 << 23, (1 << 23) + 5, MOST - 4097, MOST - 2, MOST - 1]
    return torch.tensor(at, device="cuda")


def same(a, b):
    torch = torch_mod()
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def randoms(torch, *shape):
    return torch.randint(-0x8000, 0x8000, shape, dtype=torch.int16, device="cuda") & -0x7F01 | 0x3F00   # bf16 of magnitude 0.5 to 2


@pytest.mark.parametrize("K", [16, 528])
def test_norm(K):
    torch, q = torch_mod(), Q()
    x, g = randoms(torch, MOST, K), randoms(torch, K)
    y, s = torch.empty((MOST, K), dtype=torch.int8, device="cuda"), torch.empty(MOST, device="cuda")
    q.qlin_norm_int8(x, g, y, s)
    at = rows(torch)
    y2, s2 = torch.empty((len(at), K), dtype=torch.int8, device="cuda"), torch.empty(len(at), device="cuda")
    q.qlin_norm_int8(x[at].contiguous(), g, y2, s2)
    assert same(y[at], y2) and same(s[at], s2)


def test_rope_and_cache():
    torch, q = torch_mod(), Q()
    for heads, dim in ((1, 16), (17, 64)):     # sixteen tokens to a workgroup, and one
        x, pos = randoms(torch, MOST, heads, dim), torch.arange(MOST, dtype=torch.int32, device="cuda")
        rope = q.Rope(16, interleaved=True)
        at = rows(torch)
        want = torch.empty((len(at), heads, dim), dtype=torch.int16, device="cuda")
        q.qlin_rope(x[at].contiguous(), pos[at].contiguous(), rope, want)
        if heads == 1:
            cache = q.KVCache.empty(MOST // 128, heads, 128, dim, torch.int8)
            q.qlin_cache_write(cache, pos, x, x, positions=pos, rope=rope)
            k, v = torch.zeros_like(x), torch.zeros_like(x)
            q.qlin_cache_read(cache, pos, k, v)
            few = q.KVCache.empty(1, heads, 16, dim, torch.int8)
            slots = torch.arange(len(at), dtype=torch.int32, device="cuda")
            q.qlin_cache_write(few, slots, x[at].contiguous(), x[at].contiguous(), positions=pos[at].contiguous(), rope=rope)
            k2, v2 = torch.zeros_like(want), torch.zeros_like(want)
            q.qlin_cache_read(few, slots, k2, v2)
            assert same(k[at], k2) and same(v[at], v2)
            del cache, k, v
        q.qlin_rope(x, pos, rope, x)            # in place
        assert same(x[at], want)
        del x


def test_attention():
    torch, q = torch_mod(), Q()
    S, heads, dim = 9001, 2, 32                 # three launches
    cache = q.KVCache.empty(64, 1, 16, dim, torch.bfloat16)
    cache.k.normal_()
    cache.v.normal_()
    x = torch.randn((S, heads, dim), device="cuda").bfloat16()
    table = torch.randint(0, 64, (S, 4), dtype=torch.int32, device="cuda")
    lengths = torch.randint(-1, 65, (S,), dtype=torch.int32, device="cuda")
    out, want = torch.full_like(x, 3), torch.full_like(x, 3)
    work = torch.empty(q.qlin_attn_decode_workspace(heads, cache), dtype=torch.uint8, device="cuda")
    q.qlin_attn_decode(x, cache, table, lengths, out, work)
    for i in range(0, S, 1000):
        j = slice(i, min(i + 1000, S))
        q.qlin_attn_decode(x[j], cache, table[j], lengths[j], want[j], work)
    assert same(out, want)
