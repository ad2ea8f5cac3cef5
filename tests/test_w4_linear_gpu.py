"""Projections on 4-bit weights against the 64-bit definition: every group size, zero points or none, one to four
matrices, row counts around every tile edge, odd widths and inputs that end inside a 128-input block."""
import numpy as np
import pytest

import w4_reference as R
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def pack(w):
    return Q().qlin_pack_w4(dev(w[0]), dev(w[1]), None if w[2] is None else dev(w[2]))


def outputs(M, ns, f32, guard=64):
    """Output tensors inside guarded buffers: (views, whole buffers)."""
    torch = torch_mod()
    size = 4 if f32 else 2
    raw = [torch.full((M * n * size + guard,), 0xEE, dtype=torch.uint8, device="cuda") for n in ns]
    dt = torch.float32 if f32 else torch.int16
    return [r[:M * n * size].view(dt).view(M, n) for r, n in zip(raw, ns)], raw


def check_guard(raw, guard=64):
    for r in raw:
        assert (host(r)[-guard:] == 0xEE).all(), "written past the output"


SIZES = [  # M, widths, K, group, zeros
    (1, (16,), 32, 32, False),
    (1, (1,), 128, 128, True),
    (1, (4096, 1024, 1024), 4096, 128, False),
    (1, (1000, 17), 2080, 32, True),
    (2, (48, 16, 33, 5), 192, 64, True),
    (5, (255,), 14336, 128, False),
    (15, (100,), 1056, 32, False),
    (16, (64, 200), 640, 64, True),
    (17, (130,), 384, 128, True),
    (31, (257,), 96, 32, True),
    (32, (128,), 4096, 64, False),
    (33, (77, 16), 320, 64, False),
    (63, (96,), 512, 128, False),
    (64, (300,), 160, 32, True),
    (65, (300, 40), 1152, 128, True),
    (127, (513,), 288, 32, False),
    (129, (129,), 704, 64, True),
    (200, (1024,), 128, 128, False),
    (333, (1000, 488), 2080, 32, True),
    (1025, (272,), 256, 64, False),
]


@pytest.mark.parametrize("M,ns,K,group,zeros", SIZES)
def test_exact_sums(M, ns, K, group, zeros):
    """Small integers times integer codes times powers of two: every partial sum is a multiple of 2^-3 below
    2^24 * 2^-3 (4 * 15 * K < 2^20 for K <= 14336), so f32 sums in any order are exact and the result is equal."""
    rng = np.random.default_rng([1, M, K, group])
    x = rng.integers(-4, 5, (M, K)).astype(np.float64)
    ws = [R.weights(rng, (n,), K, group, zeros, exact=True) for n in ns]
    ys, raw = outputs(M, ns, True)
    print(f"exact M={M} ns={ns} K={K} group={group} zeros={zeros}", flush=True)
    Q().qlin_linear_w4(dev(R.bf16_bits(x)), [(pack(w), y) for w, y in zip(ws, ys)], out=Q().OUT_F32)
    for w, y in zip(ws, ys):
        assert np.array_equal(host(y), R.linear(x, w, group)[0])
    check_guard(raw)


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("M,ns,K,group,zeros", SIZES)
def test_against_64_bits(M, ns, K, group, zeros, f32):
    rng = np.random.default_rng([2, M, K, group])
    xb = R.bf16_bits(rng.standard_normal((M, K)) * np.where(np.arange(K) % 97 == 0, 20.0, 1.0))
    ws = [R.weights(rng, (n,), K, group, zeros) for n in ns]
    ys, raw = outputs(M, ns, f32)
    print(f"M={M} ns={ns} K={K} group={group} zeros={zeros} f32={f32}", flush=True)
    Q().qlin_linear_w4(dev(xb), [(pack(w), y) for w, y in zip(ws, ys)], out=Q().OUT_F32 if f32 else Q().OUT_BF16)
    for w, y in zip(ws, ys):
        ref, bound = R.linear(R.bf16_values(xb), w, group)
        if f32:
            assert (np.abs(host(y) - ref) <= bound).all()
        else:
            got = R.bf16_values(host(y))
            assert (np.abs(got - ref) <= bound + R.BF16_HALF * (np.abs(ref) + bound)).all()
    check_guard(raw)


@pytest.mark.parametrize("M,I,K,group,zeros", [(1, 16, 128, 128, False), (1, 14336, 1024, 128, False), (1, 40, 2080, 32, True),
                                               (7, 129, 320, 64, True), (16, 64, 512, 32, False), (33, 200, 384, 128, True),
                                               (64, 48, 96, 32, True), (130, 260, 640, 64, False), (300, 368, 1152, 128, True)])
def test_swiglu(M, I, K, group, zeros):
    rng = np.random.default_rng([3, M, I, K])
    xb = R.bf16_bits(rng.standard_normal((M, K)) * 3)
    gate, up = (R.weights(rng, (I,), K, group, zeros) for _ in range(2))
    (h,), raw = outputs(M, [I], False)
    print(f"swiglu M={M} I={I} K={K} group={group} zeros={zeros}", flush=True)
    Q().qlin_linear_swiglu_w4(dev(xb), pack(gate), pack(up), h)
    ref, bound = R.swiglu(R.bf16_values(xb), gate, up, group)
    assert (np.abs(R.bf16_values(host(h)) - ref) <= bound + R.BF16_HALF * (np.abs(ref) + bound)).all()
    check_guard(raw)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_packed_layout_is_the_documented_one(group):
    rng = np.random.default_rng(4)
    E, N, K = 3, 37, 384 if group == 128 else 448 - 32 * (group == 32)
    codes, scales, zeros = R.weights(rng, (E, N), K, group, True)
    w = Q().qlin_pack_w4(dev(codes), dev(scales), dev(zeros))
    KT = -(-K // 128)
    q = np.zeros((E, 48, 128 * KT), np.uint8)
    q[:, :N, 0:K:2], q[:, :N, 1:K:2] = codes & 15, codes >> 4
    want = np.empty((E, 3, KT, 64, 4, 4), np.uint8)   # matrix, row tile, input block, lane, dword, byte
    for lane in range(64):
        for j in range(4):
            for b in range(4):
                k = 32 * j + 8 * (lane // 16) + b
                at = q.reshape(E, 3, 16, KT, 128)[:, :, lane % 16, :, :]
                want[:, :, :, lane, j, b] = at[..., k] | (at[..., k + 4] << 4)
    assert np.array_equal(host(w.packed), want.reshape(-1))
    for got, rows in ((host(w.scales).view(np.uint16), scales), (host(w.zeros), zeros)):
        pad = np.zeros((E, 48, KT * (128 // group)), rows.dtype)
        pad[:, :N, :K // group] = rows
        assert np.array_equal(got, pad.reshape(E, 3, 16, KT, -1).transpose(0, 1, 3, 2, 4).reshape(-1))


def test_mixed_zero_points_in_one_call():
    # one matrix with zero points beside one without
    rng = np.random.default_rng(5)
    x = rng.integers(-4, 5, (3, 256)).astype(np.float64)
    ws = [R.weights(rng, (50,), 256, 64, z, exact=True) for z in (True, False, True)]
    ys, raw = outputs(3, [50] * 3, True)
    Q().qlin_linear_w4(dev(R.bf16_bits(x)), [(pack(w), y) for w, y in zip(ws, ys)], out=Q().OUT_F32)
    for w, y in zip(ws, ys):
        assert np.array_equal(host(y), R.linear(x, w, 64)[0])
    check_guard(raw)


@pytest.mark.parametrize("M", [1, 20, 100])
def test_infinities_and_nan_stay_in_their_rows(M):
    """A row of x with an infinity or NaN gives no finite result in that row and leaves the others as they are."""
    torch = torch_mod()
    rng = np.random.default_rng(6)
    x = rng.standard_normal((M, 512))
    w = R.weights(rng, (96,), 512, 128, True)
    p = pack(w)
    xd = dev(R.bf16_bits(x))
    a, b = (torch.empty((M, 96), dtype=torch.float32, device="cuda") for _ in range(2))
    Q().qlin_linear_w4(xd, [(p, a)], out=Q().OUT_F32)
    bad = M // 2
    xd.view(torch.bfloat16)[bad, 300] = float("inf")
    xd.view(torch.bfloat16)[bad, 10] = float("nan")
    Q().qlin_linear_w4(xd, [(p, b)], out=Q().OUT_F32)
    a, b = host(a), host(b)
    assert np.isnan(b[bad]).all()
    keep = np.arange(M) != bad
    assert np.array_equal(a[keep], b[keep])


@pytest.mark.parametrize("M", [1, 40, 150])
def test_on_another_stream_and_repeated(M):
    torch = torch_mod()
    rng = np.random.default_rng(7)
    w = R.weights(rng, (512,), 1024, 128, False)
    p, x = pack(w), dev(R.bf16_bits(rng.standard_normal((M, 1024))))
    ys = [torch.empty((M, 512), dtype=torch.float32, device="cuda") for _ in range(4)]
    Q().qlin_linear_w4(x, [(p, ys[0])], out=Q().OUT_F32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    Q().qlin_linear_w4(x, [(p, ys[1])], out=Q().OUT_F32, stream=side)
    with torch.cuda.stream(side):
        Q().qlin_linear_w4(x, [(p, ys[2])], out=Q().OUT_F32)
    Q().qlin_linear_w4(x, [(p, ys[3])], out=Q().OUT_F32)       # at the same time, on the first stream
    torch.cuda.synchronize()
    for y in ys[1:]:
        assert np.array_equal(host(y), host(ys[0]))


def test_no_rows_is_a_no_op():
    torch = torch_mod()
    w = pack(R.weights(np.random.default_rng(8), (16,), 128, 128, False))
    Q().qlin_linear_w4(torch.empty((0, 128), dtype=torch.int16, device="cuda"),
                       [(w, torch.empty((0, 16), dtype=torch.int16, device="cuda"))])
