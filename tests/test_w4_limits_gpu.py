"""The largest sizes that the 4-bit, routing and experts calls take: the longest rows, the most rows of x and of a matrix, the
most slots.  Results are exact (small integers, scales that are powers of two); of large outputs the ends and a sample."""
import numpy as np
import pytest

import route_reference as RR
import w4_exact as X
import w4_reference as R
from gpu_helpers import dev, host, torch_mod
from test_experts_gpu import run
from test_w4_linear_gpu import Q, check_guard, outputs, pack

pytestmark = pytest.mark.gpu
LONGEST, MOST = 131072, 1 << 24


@pytest.fixture(autouse=True)
def free_after():
    yield
    torch_mod().cuda.empty_cache()


def sample(n):
    return np.unique(np.concatenate([[0, 1, n - 2, n - 1], np.random.default_rng(50).integers(0, n, 40)]))


@pytest.mark.parametrize("M", [1, 20, 300])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False), (64, True)])
def test_the_longest_rows(M, group, zeros):
    """x of -1..1: sums in steps of 1/8 stay below 15 * 131072 * 8 < 2^24 steps."""
    rng = np.random.default_rng([51, M, group])
    x = rng.integers(-1, 2, (M, LONGEST)).astype(np.float64)
    ws = [R.weights(rng, (n,), LONGEST, group, zeros, exact=True) for n in (40, 17)]
    ys, raw = outputs(M, [40, 17], True)
    print(f"longest rows M={M} group={group}", flush=True)
    Q().qlin_linear_w4(dev(R.bf16_bits(x)), [(pack(w), y) for w, y in zip(ws, ys)], out=Q().OUT_F32)
    for w, y in zip(ws, ys):
        assert np.array_equal(host(y), x @ R.dequantize(w)[0].T)
    check_guard(raw)


@pytest.mark.parametrize("T,H,I", [(1, LONGEST, 32), (3, 32, LONGEST), (60, LONGEST, 32), (60, 32, LONGEST)])
def test_experts_of_the_longest_rows(T, H, I):
    """As in w4_exact, with x and the down weights zero but for 256 inputs: the sums stay exact."""
    x, ids, wt, ws = X.experts_case(4, T, 2, 2, H, I, 32, True, False)
    if I == LONGEST:
        codes, _, zp = ws[2]
        keep = np.random.default_rng(52).random(I // 2) < 256 / I
        low = np.repeat(zp, 16, -1)
        codes[..., ~keep] = (low | (low << 4))[..., ~keep]          # code = zero point: weight 0
    print(f"experts T={T} H={H} I={I}", flush=True)
    y = run(R.bf16_bits(x).reshape(T, H), ids, wt, ws)
    assert np.array_equal(y, R.bf16_values(R.bf16_bits(X.experts(x, ids, wt, ws, 2))).reshape(T, H))


def test_the_most_rows_of_x():
    torch = torch_mod()
    rng = np.random.default_rng(53)
    w = R.weights(rng, (20,), 32, 32, True, exact=True)
    x = torch.randint(-4, 5, (MOST, 32), device="cuda").to(torch.bfloat16)
    y = torch.empty((MOST, 20), device="cuda")
    Q().qlin_linear_w4(x, [(pack(w), y)], out=Q().OUT_F32)
    at = torch.from_numpy(sample(MOST)).cuda()
    assert np.array_equal(host(y[at]), host(x[at].double()) @ R.dequantize(w)[0].T)


def test_the_most_rows_of_a_matrix():
    torch = torch_mod()
    gen = torch.Generator(device="cuda").manual_seed(54)
    codes = torch.randint(0, 256, (MOST, 16), dtype=torch.uint8, device="cuda", generator=gen)
    scales = torch.randint(-3, 1, (MOST, 1), device="cuda", generator=gen).exp2().to(torch.bfloat16)
    x = np.random.default_rng(54).integers(-4, 5, (3, 32)).astype(np.float64)
    w = Q().qlin_pack_w4(codes, scales)
    y = torch.empty((3, MOST), device="cuda")
    Q().qlin_linear_w4(dev(R.bf16_bits(x)), [(w, y)], out=Q().OUT_F32)
    at = torch.from_numpy(sample(MOST)).cuda()
    v = R.dequantize((host(codes[at]), R.bf16_bits(host(scales[at].float())), None))[0]
    assert np.array_equal(host(y[:, at]), x @ v.T)
    with pytest.raises(Q().QlinError):                              # one row more in all
        more = Q().qlin_pack_w4(codes[:1], scales[:1])
        Q().qlin_linear_w4(dev(R.bf16_bits(x)), [(w, y), (more, torch.empty((3, 1), device="cuda"))], out=Q().OUT_F32)


def test_the_most_tokens_routed():
    torch = torch_mod()
    logits = torch.randn((MOST, 8), device="cuda")
    ids = torch.empty((MOST, 3), dtype=torch.int32, device="cuda")
    wt = torch.empty((MOST, 3), device="cuda")
    Q().qlin_route(logits, ids, wt, score=Q().SCORE_SIGMOID, groups=4, top_groups=2)
    at = torch.from_numpy(sample(MOST)).cuda()
    rid, rw = RR.route(host(logits[at]), 3, 1, None, 4, 2)
    assert np.array_equal(host(ids[at]), rid) and (np.abs(host(wt[at]) - rw) <= 2.0 ** -23 * rw).all()


@pytest.mark.parametrize("k", [1, 32])
def test_the_most_slots(k):
    torch = torch_mod()
    T, E, H, I, group = MOST // k, 64, 32, 32, 32
    x1, _, _, ws = X.experts_case(5, 997, E, 1, H, I, group, True, False)
    gen = torch.Generator(device="cuda").manual_seed(55)
    rows = torch.arange(T, device="cuda") % 997
    x = dev(R.bf16_bits(x1).reshape(997, H))[rows].contiguous()
    ids = torch.randint(-1, E, (T, k), dtype=torch.int32, device="cuda", generator=gen)
    wt = torch.randint(-1, 2, (T, k), device="cuda", generator=gen).float().exp2()
    packed = [pack(w) for w in ws]
    y = torch.empty((T, H), dtype=torch.int16, device="cuda")
    work = torch.empty(Q().qlin_experts_w4_workspace(T, k, *packed), dtype=torch.uint8, device="cuda")
    Q().qlin_experts_w4(x, ids, wt, *packed, y, work)
    at = sample(T)
    on = torch.from_numpy(at).cuda()
    sub = (x1[at % 997], host(ids[on]), host(wt[on]))
    assert X.experts(*sub, ws, 2, magnitudes=True).max() < 16 * 2 ** 24
    assert np.array_equal(R.bf16_values(host(y[on])), R.bf16_values(R.bf16_bits(X.experts(*sub, ws, 2))).reshape(len(at), H))
    with pytest.raises(Q().QlinError):
        Q().qlin_experts_w4_workspace(T + 1, k, *packed)
