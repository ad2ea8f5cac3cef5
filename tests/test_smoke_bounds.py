"""The bound of the smoke pass's attention refuses wrong outputs (planted here, on the CPU) and takes the rounded right one."""
import numpy as np
import pytest

import __graft_entry__ as entry
import oracle as O


@pytest.fixture(scope="module")
def step():
    c = entry.smoke_tokens()
    rows = []
    for n in ("k", "v"):
        x = O.bf16_bits_to_f64(c[n])
        scale = np.abs(x).max(-1, keepdims=True) / 448
        rows.append(O.e4m3_decode(O.e4m3_encode((x / scale).astype(np.float32))) * scale)
    return O.bf16_bits_to_f64(c["q"])[0], *rows


def refused(y, step):
    """-> for each head, whether its output is refused."""
    ref, room = entry.smoke_attention(*step)
    return (np.abs(O.bf16_bits_to_f64(O.round_to_bf16_bits(y)) - ref) > room).any(-1)


def test_the_right_output_is_taken(step):
    assert not refused(entry.smoke_attention(*step)[0], step).any()


def test_wrong_outputs_are_refused_in_every_head(step):
    q, k, v = step
    heads, kv = q.shape[0], k.shape[1]
    of = lambda *a: entry.smoke_attention(*a)[0]     # noqa: E731
    wrong = {
        "zeros": np.zeros(q.shape),
        "mean of the values": v.mean(0)[np.arange(heads) * kv // heads],
        "the other kv head": of(q, k[:, ::-1], v[:, ::-1]),
        "keys and values of different heads": of(q, k, v[:, ::-1]),
        "the next head's": np.roll(of(*step), 1, 0),
        "no softmax scale": of(q * 8, k, v),
        "half of the softmax scale": of(q / 2, k, v),
        "without the first page": of(q, k[16:], v[16:]),
        "pages in another order": of(q, k, np.concatenate([v[16:32], v[:16], v[32:]])),
    }
    for name, y in wrong.items():
        assert refused(y, step).all(), (name, refused(y, step))
    tail = refused(of(q, k[:-8], v[:-8]), step)      # the last, partial page: its tokens may weigh nothing in some heads
    assert tail.any()
