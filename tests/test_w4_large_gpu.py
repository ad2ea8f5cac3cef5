"""Offsets past 32 bits: outputs, logits and experts' weights of more than 4 GiB, checked where they pass 2^31 and 2^32
and at their ends.  And zero points past the codes' range."""
import numpy as np
import pytest

import w4_reference as R
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


@pytest.fixture(autouse=True)
def free_after():
    yield
    torch_mod().cuda.empty_cache()


def rows_around(row_bytes, total):
    """Rows at the start, where the byte and element offsets pass 2^31 and 2^32, and at the end."""
    at = {0, 1, total - 2, total - 1}
    for limit in (2 ** 31, 2 ** 32, 2 ** 33):
        r = limit // row_bytes
        at |= {t for t in (r - 1, r, r + 1) if 0 <= t < total}
    return np.array(sorted(at))


def test_outputs_past_32_bits():
    torch = torch_mod()
    M, N, K, group = 270001, 16400, 32, 32
    rng = np.random.default_rng(21)
    w = R.weights(rng, (N,), K, group, True)
    xb = R.bf16_bits(rng.standard_normal((M, K)))
    y = torch.empty((M, N), dtype=torch.int16, device="cuda")
    Q().qlin_linear_w4(dev(xb), [(Q().qlin_pack_w4(*(dev(t) for t in w)), y)])
    at = rows_around(2 * N, M)
    got = R.bf16_values(host(y[torch.from_numpy(at).cuda()]))
    ref, bound = R.linear(R.bf16_values(xb[at]), w, group)
    assert (np.abs(got - ref) <= bound + R.BF16_HALF * (np.abs(ref) + bound)).all()


def test_logits_past_32_bits():
    torch = torch_mod()
    T, E, k = 1 << 24, 160, 3
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_()
    ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
    wt = torch.empty((T, k), device="cuda")
    Q().qlin_route(logits, ids, wt)
    at = rows_around(2 * E, T)
    sel = torch.from_numpy(at).cuda()
    ref_ids, ref_wt = R.route(host(logits[sel].float()), k, 0, None, 1, 1, 2, True, 1.0)
    assert np.array_equal(host(ids[sel]), ref_ids)
    assert (np.abs(host(wt[sel]) - ref_wt) <= 2 * R.U * ref_wt).all()


@pytest.mark.parametrize("T", [2, 300, 9000])
def test_experts_weights_past_32_bits(T):
    """One token after the other, streamed, and tiled."""
    torch = torch_mod()
    q = Q()
    E, H, I, group, k = 1024, 2048, 4224, 64, 2
    gen = torch.Generator(device="cuda").manual_seed(22)

    def weight(N, K):
        codes = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
        scales = torch.empty((E, N, K // group), dtype=torch.bfloat16, device="cuda").uniform_(1e-3, 5e-3, generator=gen)
        return codes, scales
    used = np.array([0, 511, 512, 1022, 1023])      # 4.4 MiB of codes each: byte 2^31 lies in expert 496, 2^32 in 992
    raw = [weight(I, H), weight(I, H), weight(H, I)]
    packed = [q.qlin_pack_w4(*w) for w in raw]
    sel = torch.from_numpy(used).cuda()
    few = [(host(c[sel]), host(s[sel].view(torch.int16)), None) for c, s in raw]
    del raw
    rng = np.random.default_rng([23, T])
    xb = R.bf16_bits(rng.standard_normal((T, H)))
    which = np.stack([rng.permutation(len(used))[:k] for _ in range(T)])
    wt = rng.random((T, k)).astype(np.float32)
    y = torch.empty((T, H), dtype=torch.int16, device="cuda")
    work = torch.empty(q.qlin_experts_w4_workspace(T, k, *packed), dtype=torch.uint8, device="cuda")
    q.qlin_experts_w4(dev(xb), dev(used[which].astype(np.int32)), dev(wt), *packed, y, work)
    at = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 10)]))
    got = R.bf16_values(host(y[torch.from_numpy(at).cuda()]))
    ref, bound = R.experts(R.bf16_values(xb[at]), which[at], wt[at], *few, group)
    assert (np.abs(got - ref) <= bound + R.BF16_HALF * (np.abs(ref) + bound)).all()


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_zero_points_of_eight_bits(M, group):
    torch = torch_mod()
    N, K = 130, 384
    rng = np.random.default_rng([24, M, group])
    codes, scales, zeros = R.weights(rng, (N,), K, group, True)
    zeros = rng.choice(np.array([0, 16, 127, 128, 254, 255], np.uint8), zeros.shape)
    xb = R.bf16_bits(rng.standard_normal((M, K)))
    y = torch.empty((M, N), device="cuda")
    Q().qlin_linear_w4(dev(xb), [(Q().qlin_pack_w4(dev(codes), dev(scales), dev(zeros)), y)], out=Q().OUT_F32)
    ref, bound = R.linear(R.bf16_values(xb), (codes, scales, zeros), group)
    assert (np.abs(host(y) - ref) <= bound).all()
