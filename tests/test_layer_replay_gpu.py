"""The norm, rotary, cache and attention calls captured once and replayed on other inputs, with eager calls between the
replays; on streams of their own; and two graphs at once, each with its workspace.  Equality bit for bit throughout."""
import numpy as np
import pytest

import layer_reference as R
from gpu_helpers import dev, torch_mod
from test_attn_gpu import Case

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def capture(torch, step):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    return graph


def bits(rng, *shape):
    return dev(R.bits(rng.standard_normal(shape)))


def replays(torch, step, inputs, outputs, changes, poison):
    """step captured; for each change of the inputs: a replay and an eager call (in turn first) give the same bits."""
    graph = capture(torch, step)
    for n, change in enumerate(changes):
        for t, value in zip(inputs, change):
            t.copy_(value)
        got = []
        for run in ((graph.replay, step) if n % 2 == 0 else (step, graph.replay)):
            poison()
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            got.append([o.clone() for o in outputs])
        for a, b in zip(*got):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
    return got


@pytest.mark.parametrize("kind", ["int8", "block", "bf16"])
@pytest.mark.parametrize("M,K", [(1, 4096), (33, 1408), (2, 40960)])
def test_norm(kind, M, K):
    torch, q = torch_mod(), Q()
    rng = np.random.default_rng(M)
    x, r, g = bits(rng, M, K), bits(rng, M, K), bits(rng, K)
    total = torch.empty_like(x)
    y = torch.empty((M, K), dtype=torch.int16 if kind == "bf16" else torch.int8, device="cuda")
    s = torch.empty((M, K // 128) if kind == "block" else (M,), device="cuda")

    def step():
        if kind == "bf16":
            q.qlin_norm_bf16(x, g, y, residual=r, sum_out=total)
        elif kind == "int8":
            q.qlin_norm_int8(x, g, y, s, residual=r, sum_out=total)
        else:
            q.qlin_norm_fp8(x, g, y, s, group=128, residual=r, sum_out=total)

    def poison():
        y.fill_(3), total.fill_(3), s.fill_(3)
    replays(torch, step, [x, r], [y, total, s], [(bits(rng, M, K), bits(rng, M, K)) for _ in range(4)], poison)


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8"])
def test_cache_write_and_read(kind):
    torch, q = torch_mod(), Q()
    rng = np.random.default_rng(2)
    T, heads, kv, dim, page, pages = 9, 8, 2, 128, 16, 3
    cache = q.KVCache.empty(pages, kv, page, dim, {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[kind])
    rope = q.Rope(dim, 5e5)
    qkv, positions = bits(rng, T, heads + 2 * kv, dim), dev(rng.integers(0, 9999, T).astype(np.int32))
    slots = dev(rng.permutation(pages * page)[:T].astype(np.int32))
    parts = qkv.split((heads, kv, kv), 1)
    out = torch.empty((T, heads, dim), dtype=torch.int16, device="cuda")
    k, v = (torch.empty((T, kv, dim), dtype=torch.int16, device="cuda") for _ in range(2))
    outputs = [out, k, v] + [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]

    def step():
        q.qlin_cache_write(cache, slots, parts[1], parts[2], positions=positions, rope=rope, q=parts[0], q_out=out)
        q.qlin_cache_read(cache, slots, k, v)

    def poison():
        for t in outputs:
            t.view(torch.uint8).fill_(7)
    changes = []
    for i in range(4):
        at = rng.permutation(pages * page)[:T].astype(np.int32)
        if i == 2:
            at[::2] = -1
        changes.append((bits(rng, T, heads + 2 * kv, dim), dev(rng.integers(0, 9999, T).astype(np.int32)), dev(at)))
    replays(torch, step, [qkv, positions, slots], outputs, changes, poison)


def attention(c, q, out, work, table, lengths, stream=None):
    return lambda: Q().qlin_attn_decode(q, c.cache, table, lengths, out, work, stream=stream)


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8"])
@pytest.mark.parametrize("columns", [16, 300])     # one launch, or two
def test_attention_replayed_at_other_lengths(kind, columns):
    """The launches do not go by the lengths: long ones, short ones, none, and rows that hold no sequence."""
    torch = torch_mod()
    c = Case(21, kind, [240, 100, 17, 1, 60], 8, 2, 64, 16, columns=columns).load()
    rng = np.random.default_rng(5)
    q, table, lengths = dev(c.q), dev(c.table), dev(c.lengths)
    out = torch.empty(c.q.shape, dtype=torch.int16, device="cuda")
    work = torch.empty(Q().qlin_attn_decode_workspace(8, c.cache), dtype=torch.uint8, device="cuda")
    changes = []
    for new in ([1, 16, 240, 7, 33], [0, 0, 0, 0, 0], [-1, 240, -1, 0, 5], [columns * 16, 100, columns * 16, 300, 2], [240, 100, 17, 1, 60]):
        pages = rng.integers(-1, c.pages, c.table.shape).astype(np.int32)
        changes.append((dev(R.bits(rng.standard_normal(c.q.shape))), dev(pages), dev(np.array(new, np.int32))))
    changes.append((dev(c.q), dev(c.table), dev(c.lengths)))

    def poison():
        out.fill_(0x1234), work.fill_(0xEE)
    last = replays(torch, attention(c, q, out, work, table, lengths), [q, table, lengths], [out], changes, poison)
    c.check(last[0][0].cpu().numpy())


def test_calls_on_a_stream_of_their_own():
    """A stream given by handle or object is the one that is used: the null stream is kept busy, and its input changes."""
    torch, q = torch_mod(), Q()
    c = Case(22, "int8", [500, 33, 1000], 8, 2, 64, 16).load()
    want = c.run()
    side = torch.cuda.Stream()
    for given in (side, side.cuda_stream):
        assert np.array_equal(want, c.run(stream=given))
    x, g = bits(np.random.default_rng(1), 64, 4096), bits(np.random.default_rng(2), 4096)
    y, s = torch.empty((64, 4096), dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda")
    y2, s2 = torch.empty_like(y), torch.empty_like(s)
    q.qlin_norm_int8(x, g, y, s)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        q.qlin_norm_int8(x, g, y2, s2)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(s, s2)


def test_two_graphs_at_once():
    """Each with a workspace of its own, on two streams; then both on one, one after the other, sharing one."""
    torch = torch_mod()
    cases = [Case(23 + i, "fp8", [3000 + 500 * i, 77, 900], 8, 2, 128, 64).load() for i in range(2)]
    held = []
    for shared in (False, True):
        parts = []
        for i, c in enumerate(cases):
            q, table, lengths = dev(c.q), dev(c.table), dev(c.lengths)
            out = torch.empty(c.q.shape, dtype=torch.int16, device="cuda")
            work = held[0] if shared and held else torch.empty(Q().qlin_attn_decode_workspace(8, c.cache), dtype=torch.uint8, device="cuda")
            held.append(work)
            parts.append((capture(torch, attention(c, q, out, work, table, lengths)), out, (q, table, lengths)))
        streams = [torch.cuda.Stream() for _ in range(2)]
        for rep in range(5):
            for _, out, _ in parts:
                out.fill_(0x1234)
            torch.cuda.synchronize()
            for i, (graph, _, _) in enumerate(parts):
                with torch.cuda.stream(streams[0 if shared else i]):
                    graph.replay()
            torch.cuda.synchronize()
            for c, (_, out, _) in zip(cases, parts):
                c.check(out.cpu().numpy())


@pytest.mark.parametrize("kind", ["bf16", "int8", "fp8"])
def test_calls_without_rows(kind):
    """No tokens, rows or sequences (torch gives such tensors a null address): nothing is written and nothing fails.  A page
    table without columns: zeros, and rows of a negative length stay."""
    torch, q = torch_mod(), Q()
    dtype = {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[kind]
    def none(*shape, dtype=torch.int16):
        return torch.empty(shape, dtype=dtype, device="cuda")
    ints = none(0, dtype=torch.int32)
    cache = q.KVCache.empty(2, 2, 16, 64, dtype)
    stored = [t for t in (cache.k, cache.v, cache.k_scale, cache.v_scale) if t is not None]
    for t in stored:
        t.view(torch.uint8).fill_(0x5A)
    rope = q.Rope(64)
    gamma = torch.zeros(64, dtype=torch.int16, device="cuda")
    wide = torch.zeros(256, dtype=torch.int16, device="cuda")
    codes, scales = none(0, 256, dtype=torch.int8), none(0, dtype=torch.float32)
    q.qlin_norm_bf16(none(0, 256), wide, none(0, 256), residual=none(0, 256), sum_out=none(0, 256))
    q.qlin_norm_int8(none(0, 256), wide, codes, scales)
    q.qlin_norm_fp8(none(0, 256), wide, codes, scales)
    q.qlin_norm_fp8(none(0, 256), wide, codes, none(0, 2, dtype=torch.float32), group=128)
    q.qlin_rope(none(0, 4, 64), ints, rope, none(0, 4, 64), gamma=gamma)
    q.qlin_cache_write(cache, ints, none(0, 2, 64), none(0, 2, 64), positions=ints, rope=rope, q=none(0, 4, 64), q_out=none(0, 4, 64),
                       q_gamma=gamma, k_gamma=gamma)
    q.qlin_cache_read(cache, ints, none(0, 2, 64), none(0, 2, 64))
    work = none(q.qlin_attn_decode_workspace(4, cache), dtype=torch.uint8)
    q.qlin_attn_decode(none(0, 4, 64), cache, none(0, 3, dtype=torch.int32), ints, none(0, 4, 64), work)
    out = torch.full((3, 4, 64), 0x5A5A, dtype=torch.int16, device="cuda")
    lengths = torch.tensor([7, -1, 0], dtype=torch.int32, device="cuda")
    q.qlin_attn_decode(torch.zeros_like(out), cache, none(3, 0, dtype=torch.int32), lengths, out, work)
    torch.cuda.synchronize()
    assert not out[0].any() and bool((out[1] == 0x5A5A).all()) and not out[2].any()
    for t in stored:
        assert bool((t.view(torch.uint8) == 0x5A).all())
