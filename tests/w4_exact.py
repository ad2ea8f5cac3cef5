"""Inputs of the gated products whose results are exact: every sum a multiple of a power of two that f32 holds, gates
of 20 or more (silu(g) = g in f32: 1 + e^-20 rounds to 1), so that equality can be asked for (NumPy)."""
import numpy as np

import w4_reference as R


def swiglu_case(seed, M, I, K, group, zeros):
    """x [M, K], gate and up [I, K]: input 0 is 256 and has gate weight 7 or 8, the others are small beside it."""
    rng = np.random.default_rng([seed, M, I, K])
    x = rng.integers(-2, 3, (M, K)).astype(np.float64)
    x[:, 0] = 256
    gate, up = (R.weights(rng, (I,), K, group, zeros, exact=True) for _ in range(2))
    codes, scales, zp = gate
    if zeros:
        zp[:, 0] = rng.integers(0, 8, I)
        codes[:, 0] = (codes[:, 0] & 0xF0) | (zp[:, 0] + 8 - rng.integers(0, 2, I)).astype(np.uint8)
    else:
        codes[:, 0] = (codes[:, 0] & 0xF0) | 15
    scales[:, 0] = R.bf16_bits(np.ones(1))[0]
    return x, gate, up


def swiglu(x, gate, up):
    """h in f32 (one rounding of the product of two exact sums), and the gates."""
    g, u = x @ R.dequantize(gate)[0].T, x @ R.dequantize(up)[0].T
    return g.astype(np.float32) * u.astype(np.float32), g


def _encode(v, zp):
    """Integer weights [.., N, K] and zero points [.., N, groups] -> codes."""
    c = v + np.repeat(zp, v.shape[-1] // zp.shape[-1], -1)
    assert c.min() >= 0 and c.max() <= 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def experts_case(seed, T, E, k, H, I, group, zeros, low):
    """Tokens with 16, 64..72 and 1 in three inputs; gate rows take the first (g = 64 or 128), up rows the second (a multiple of 4
    from 256 to 504).  low: rows come in pairs, the odd one also takes the third input, so that u is 4 m and 4 m + 1, which one
    bf16 tells apart no more (a tie, to the even 4 m); the down weights of a pair are -v and v, so that the result is what the
    one bf16 of h leaves out, g v per pair.  Otherwise h is a bf16 number and the down weights are any."""
    rng = np.random.default_rng([seed, T, E, H, I])
    x = rng.integers(-3, 4, (T, H)).astype(np.float64)
    a, b, c = rng.permutation(H)[:3]
    x[:, a], x[:, b], x[:, c] = 16, rng.choice([64, 68, 72], T), 1

    def scales(n, K, of):
        return R.bf16_bits(2.0 ** rng.integers(*of, (E, n, K // group)))

    def zeros_of(n, K, lo, hi):
        return rng.integers(lo, hi, (E, n, K // group)) if zeros else np.full((E, n, K // group), 8)

    def weight(v, s, zp):
        return _encode(v, zp), s, zp.astype(np.uint8) if zeros else None
    gate, up = np.zeros((E, I, H), np.int64), np.zeros((E, I, H), np.int64)
    gate[:, :, a] = 4
    up[:, :, b] = rng.integers(4, 8, (E, I))
    gs, us = scales(I, H, (-1, 2)), scales(I, H, (-1, 2))
    gs[:, :, a // group] = R.bf16_bits(2.0 ** rng.integers(0, 2, (E, I)))
    one = R.bf16_bits(np.ones(1))[0]
    us[:, :, b // group] = us[:, :, c // group] = one
    if low:
        up[:, 1::2, b] = up[:, 0::2, b]
        up[:, 1::2, c] = 1
        gs[:, 1::2] = gs[:, 0::2]
        v = rng.integers(-4, 5, (E, H, I // 2))
        down = np.stack([-v, v], -1).reshape(E, H, I)
    else:
        down = rng.integers(-4, 5, (E, H, I))
    ws = [weight(gate, gs, zeros_of(I, H, 0, 9)), weight(up, us, zeros_of(I, H, 0, 9)),
          weight(down, scales(H, I, (-1, 1)), zeros_of(H, I, 4, 12))]
    ids = np.argsort(rng.random((T, E)), 1)[:, :k].astype(np.int32)
    wt = (2.0 ** rng.integers(-1, 2, (T, k))).astype(np.float32)
    return x, ids, wt, ws


def experts(x, ids, wt, ws, parts, magnitudes=False):
    """y in 64 bits, h kept as a sum of `parts` bf16 numbers; or the sum of its terms' magnitudes."""
    y = np.zeros_like(x)
    for e in range(len(ws[0][0])):           # any other id: no expert
        token, slot = np.nonzero(ids == e)
        g, u = (x[token] @ R.dequantize(tuple(None if t is None else t[e] for t in w))[0].T for w in ws[:2])
        left, h = g * u, np.zeros_like(g)
        for _ in range(parts):
            part = R.bf16_values(R.bf16_bits(left)).reshape(g.shape)
            h, left = h + part, left - part
        v = R.dequantize(tuple(None if t is None else t[e] for t in ws[2]))[0]
        np.add.at(y, token, wt[token, slot][:, None].astype(np.float64) * (h @ (np.abs(v) if magnitudes else v).T))
    return y


LOW = [  # T, E, k, H, I, group, zeros: few rows of each expert
    (1, 16, 4, 256, 512, 128, False), (2, 8, 2, 128, 256, 128, True), (4, 6, 3, 128, 160, 32, True), (30, 24, 4, 256, 320, 64, True),
    (64, 65, 8, 128, 256, 64, False), (90, 12, 2, 128, 256, 128, False), (129, 256, 4, 128, 256, 32, True),
]
ANY = LOW + [(70, 3, 2, 128, 128, 128, False), (130, 2, 1, 192, 320, 64, True), (300, 4, 2, 640, 384, 128, False), (400, 7, 7, 128, 128, 32, True),
             (600, 300, 3, 64, 64, 64, True), (900, 3, 3, 256, 160, 32, False)]
MANY = [  # many rows of each expert: the streaming forms of more rows, and the tiled ones
    (300, 3, 3, 256, 128, 32, True), (1000, 3, 3, 128, 128, 64, True), (1000, 2, 2, 256, 128, 128, True), (700, 2, 2, 256, 128, 32, False),
    (2500, 3, 3, 128, 128, 128, True), (3000, 3, 3, 256, 128, 128, False), (2500, 3, 3, 128, 256, 128, True), (2000, 3, 3, 256, 128, 64, False),
    (3000, 3, 3, 512, 256, 64, True), (2000, 9, 3, 256, 128, 32, True), (2000, 4, 3, 1024, 512, 32, True),
]
ANY += MANY
SWIGLU = [  # M, I, K, group, zeros
    (1, 16, 128, 128, False), (1, 4096, 1024, 128, True), (1, 40, 2080, 32, True), (7, 129, 320, 64, True), (16, 64, 512, 32, False),
    (33, 200, 384, 128, True), (64, 48, 96, 32, True), (130, 260, 640, 64, False), (300, 368, 1152, 128, True), (700, 1000, 256, 32, True),
    (2048, 512, 128, 64, False),
]
