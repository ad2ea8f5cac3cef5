"""The norm calls against their definition: the residual sum and the codes bit for bit (every step up to them is one IEEE
operation), the scales and the bf16 values within the derived bounds."""
import numpy as np
import pytest

import layer_reference as R
import oracle as O
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def guarded(torch, nbytes):
    raw = torch.full((nbytes + 64,), 0xEE, dtype=torch.uint8, device="cuda")
    return raw, raw[:nbytes]


def run(kind, xb, rb, gb, eps=1e-6, in_place=False, stream=None):
    """-> (sum bits or None, codes' or bf16 values, scales or None)"""
    torch, q = torch_mod(), Q()
    M, K = xb.shape
    x, g = dev(xb), dev(gb)
    r = None if rb is None else dev(rb)
    total, total_raw = None, None
    if r is not None:
        if in_place:
            total = r
        else:
            total_raw, t = guarded(torch, 2 * M * K)
            total = t.view(torch.int16).view(M, K)
    more = dict(residual=r, sum_out=total, eps=eps, stream=stream)
    bytes_out = M * K * (2 if kind == "bf16" else 1)
    y_raw, y = guarded(torch, bytes_out)
    groups = (M, K // 128) if kind == "block" else (M,)
    s_raw, s = guarded(torch, 4 * int(np.prod(groups)))
    s = s.view(torch.float32).view(groups)
    if kind == "bf16":
        y = y.view(torch.int16).view(M, K)
        q.qlin_norm_bf16(x, g, y, **more)
    elif kind == "int8":
        y = y.view(torch.int8).view(M, K)
        q.qlin_norm_int8(x, g, y, s, **more)
    else:
        y = y.view(M, K)
        q.qlin_norm_fp8(x, g, y, s, group=128 if kind == "block" else 0, **more)
    torch.cuda.synchronize()
    for raw in (y_raw, s_raw, total_raw):
        assert raw is None or (host(raw)[-64:] == 0xEE).all(), "written past a buffer"
    if kind == "bf16":
        return None if total is None else host(total), R.value(host(y)), None
    codes = host(y).astype(np.float64) if kind == "int8" else O.e4m3_decode(host(y))
    return None if total is None else host(total), codes, host(s)


def check(kind, xb, rb, gb, got, eps=1e-6):
    total, y, s = got
    M, K = xb.shape
    row = xb
    if rb is not None:
        row = R.residual_sum(xb, rb)
        assert np.array_equal(total.view(np.uint16), row), "residual sum"
    t, d = R.norm(row, gb, eps)
    slack = R.norm_slack(K)
    if kind == "bf16":
        ref = t * d[:, None]
        assert (np.abs(y - ref) <= np.abs(ref) * (R.HALF * (1 + slack) + slack) + 1e-40).all()
        return
    rows = t.reshape(M, -1, 128) if kind == "block" else t
    want, a = R.codes(rows, "int8" if kind == "int8" else "fp8")
    assert np.array_equal(y, want.reshape(M, K)), "codes"
    # s = f32(absmax) * d / Q: the reference's a is absmax / Q
    ref = a.astype(np.float64) * (d[:, None] if kind == "block" else d)
    assert (np.abs(s - ref) <= np.abs(ref) * (slack + 4 * R.U32) + 1e-44).all()


def inputs(seed, M, K, residual=True):
    rng = np.random.default_rng([seed, M, K])
    gain = np.where(np.arange(K) % 37 == 5, 20.0, 1.0)
    xb = R.bits(rng.standard_normal((M, K)) * gain)
    rb = R.bits(2 * rng.standard_normal((M, K))) if residual else None
    return xb, rb, R.bits(1 + 0.2 * rng.standard_normal(K))


KINDS = ["bf16", "int8", "fp8", "block"]
SIZES = [(1, 16), (3, 48), (5, 128), (7, 512), (2, 528), (9, 640), (1, 2048), (33, 2064), (1, 4096), (17, 4096), (3, 4112), (2, 8192), (2, 8208),
         (3, 14336), (1, 32768), (2, 32784), (1, 65552), (2, 65664), (1, 131072), (513, 256), (1025, 1408)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("M,K", SIZES)
def test_norm(kind, M, K):
    if kind == "block" and K % 128:
        K = K // 128 * 128 + 128
    for residual in (False, True):
        case = inputs(1, M, K, residual)
        check(kind, *case, run(kind, *case))


@pytest.mark.parametrize("kind", KINDS)
def test_residual_updated_in_place(kind):
    for M, K in ((21, 1024), (2, 40960)):
        case = inputs(2, M, K)
        check(kind, *case, run(kind, *case, in_place=True))


@pytest.mark.parametrize("kind", KINDS)
def test_special_rows(kind):
    """Rows of zeros, of tiny and of large values, one live input, gammas of zero; each next to ordinary rows."""
    xb, rb, gb = inputs(3, 12, 256, False)
    x = R.value(xb).copy()
    x[1] = 0
    x[3] *= 2.0 ** -70
    x[4] *= 2.0 ** 50 / 16
    x[5] = 0
    x[5, 200] = -3.0
    x[7, :128] = 0
    x[9] = x[8]
    xb = R.bits(x)
    check(kind, xb, None, gb, run(kind, xb, None, gb))
    g = R.value(gb).copy()
    g[:128] = 0
    g[130] = -2
    check(kind, xb, None, R.bits(g), run(kind, xb, None, R.bits(g)))
    check(kind, xb, None, gb, run(kind, xb, None, gb, eps=1e-20), eps=1e-20)
    check(kind, xb, None, gb, run(kind, xb, None, gb, eps=0.5), eps=0.5)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_are_not_finite_stay_alone(kind):
    xb, _, gb = inputs(4, 9, 512, False)
    bad = xb.copy()
    bad[2, 5], bad[4, 6], bad[8, 511] = 0x7F80, 0x7FC0, 0xFF80
    good = [0, 1, 3, 5, 6, 7]
    total, y, s = run(kind, bad, None, gb)
    check(kind, xb[good], None, gb, (None, y[good], None if s is None else s[good]))


def test_codes_beside_those_of_the_quantizers():
    """With gamma 1 the codes are those that the activation quantizers give for the row itself, but where the last bit of
    the reciprocal decides: two codes that differ are neighbours, and the value is their border to f32's precision (three
    roundings on either side).  s is theirs times d."""
    torch, q = torch_mod(), Q()
    xb, _, _ = inputs(5, 40, 4096, False)
    ones = np.full(4096, 0x3F80, np.uint16)
    for kind, group in (("int8", None), ("fp8", 0), ("block", 128)):
        qx = torch.empty((40, 4096), dtype=torch.uint8, device="cuda")
        sx = torch.empty((40, 32) if kind == "block" else (40,), device="cuda")
        if kind == "int8":
            q.qlin_quant_act_int8(dev(xb), qx, sx)
        else:
            q.qlin_quant_act_fp8(dev(xb), qx, sx, group=group)
        _, codes, s = run(kind, xb, None, ones)
        raw = host(qx)
        theirs = raw.view(np.int8).astype(np.float64) if kind == "int8" else O.e4m3_decode(raw)
        x = R.value(xb).reshape(40, -1, 128 if kind == "block" else 4096)
        v = (x * (127.0 if kind == "int8" else 448.0) / np.abs(x).max(-1, keepdims=True)).reshape(40, 4096)
        other = codes != theirs
        assert (np.abs(v - (codes + theirs) / 2)[other] <= 4 * R.U32 * np.abs(v)[other]).all()
        _, d = R.norm(xb, ones, 1e-6)
        ref = host(sx) * (d[:, None] if kind == "block" else d)
        assert (np.abs(s - ref) <= np.abs(ref) * (R.norm_slack(4096) + 4 * R.U32)).all()


@pytest.mark.parametrize("kind", ["int8", "fp8", "block"])
def test_codes_equal_an_evaluation_in_torch(kind):
    """Bit for bit, over a million values."""
    torch, q = torch_mod(), Q()
    xb, rb, gb = inputs(7, 300, 4096)
    _, codes, _ = run(kind, xb, rb, gb)
    r = (dev(xb).view(torch.bfloat16).float() + dev(rb).view(torch.bfloat16).float()).bfloat16().float()
    t = r * dev(gb).view(torch.bfloat16).float()
    t = t.view(300, -1, 128) if kind == "block" else t
    most = 127.0 if kind == "int8" else 448.0
    v = t * (most / t.abs().amax(-1, keepdim=True))
    v = v.round() if kind == "int8" else v.clamp(-448, 448).to(torch.float8_e4m3fn).float()
    assert np.array_equal(codes, host(v.reshape(300, 4096)).astype(np.float64))


def test_many_rows_and_long_offsets():
    """More than 2^31 elements: the last rows are right."""
    torch, q = torch_mod(), Q()
    M, K = (1 << 31) // 16384 + 40, 16384
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(-0x4000, 0x4000, (64, K), generator=g, dtype=torch.int16, device="cuda")   # any bit patterns: compared as bits
    big = torch.zeros((M, K), dtype=torch.int16, device="cuda")
    big[-64:] = x
    gamma = dev(inputs(6, 1, K)[2])
    y = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    s = torch.empty((M, K // 128), device="cuda")
    q.qlin_norm_fp8(big, gamma, y, s, group=128)
    y2, s2 = torch.empty((64, K), dtype=torch.uint8, device="cuda"), torch.empty((64, K // 128), device="cuda")
    q.qlin_norm_fp8(x, gamma, y2, s2, group=128)
    assert torch.equal(y[-64:], y2) and torch.equal(s[-64:].view(torch.int32), s2.view(torch.int32)) and int(y[:-64].count_nonzero()) == 0
