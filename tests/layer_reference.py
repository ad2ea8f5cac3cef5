"""The norm, rotary, cache and attention calls in 64 bits on the CPU, from their definitions, with bounds on the error
of an f32 evaluation.  Test infrastructure; shares no code with the library."""
import numpy as np

import oracle as O

HALF = 2.0 ** -8          # half a step of bf16, relative
U32 = 2.0 ** -24          # half a step of f32, relative
MOST = {"int8": 127.0, "fp8": 448.0}


def bits(a):
    """The nearest bf16 (bits) of an array."""
    return O.round_to_bf16_bits(np.asarray(a, np.float64)).astype(np.uint16)


def value(b):
    return O.bf16_bits_to_f64(np.asarray(b).view(np.uint16))


# ---- norm -----------------------------------------------------------------

def residual_sum(xb, rb):
    """bf16(f32(x + residual)) as bits."""
    s = value(xb).astype(np.float32) + value(rb).astype(np.float32)
    return bits(s)


def norm(rb, gb, eps):
    """rows (bits) -> (t = r * gamma, exact in f32; d, in f64)."""
    r, g = value(rb), value(gb)
    return r * g, 1 / np.sqrt((r * r).mean(1) + eps)


def norm_slack(K):
    """Relative error of d in f32: a lane adds up to K / 512 + 8 squares one after the other (16 chunks of 8 at most),
    6 levels of lanes and 16 wavefronts; d takes half of the sum's, and a division, an addition, a root, a division and
    a product follow, two units each at most."""
    return U32 * ((min(K, 128) + 22) / 2 + 12)


def codes(t, kind):
    """t f32 [..., n] -> (codes as the values they stand for, scales), step by step in f32 as the header defines it."""
    t = t.astype(np.float32)
    a = np.abs(t).max(-1, keepdims=True)
    q = np.float32(MOST[kind])
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        pre = np.where(a < np.float32(2.0 ** -64), np.float32(2.0 ** 64), np.float32(1))
        inv = np.where(a == 0, np.float32(0), q * (np.float32(1) / (a * pre))).astype(np.float32)
    v = np.clip(((t * pre).astype(np.float32) * inv).astype(np.float32), -q, q)
    # (+ 0.0: integers have no minus zero)
    c = np.rint(v) + 0.0 if kind == "int8" else O.e4m3_decode(O.e4m3_encode(v))
    return c.astype(np.float64), (a / q)[..., 0].astype(np.float32)


# ---- rotation -------------------------------------------------------------

def rotate(x, positions, frequencies, dims, interleaved, strength, gamma=None, eps=1e-6):
    """x f64 [T, heads, dim] -> (y, bound of an f32 evaluation's error before y is rounded)."""
    slack = np.zeros_like(x)
    if gamma is not None:
        d = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x = x * gamma * d
        slack = np.abs(x) * U32 * 60       # 8 products in a lane, 5 levels, root and divisions, two products
    angle = positions.astype(np.float64)[:, None] * frequencies[None]
    c, s = np.cos(angle)[:, None] * strength, np.sin(angle)[:, None] * strength
    half = dims // 2
    i = np.arange(half)
    first, second = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = x[..., first], x[..., second]
    y, e = x.copy(), slack.copy()
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    # the reduced angle (at most pi) is rounded to f32: 2^-23; its sine and cosine are off by two units more
    room = (np.abs(a) + np.abs(b)) * strength * (2.0 ** -21) + (slack[..., first] + slack[..., second]) * strength
    e[..., first], e[..., second] = room, room
    return y, e


# ---- attention ------------------------------------------------------------

def attention(q, k, v, pages, lengths, page_size, window, scale):
    """q f64 [S, heads, dim]; k, v f64 [pages, kv_heads, page_size, dim] (masked places may hold anything) ->
    (out, bound before rounding); out is NaN where a row has to stay as it was."""
    S, heads, dim = q.shape
    kv_heads = k.shape[1]
    out, room = np.zeros(q.shape), np.zeros(q.shape)
    for s in range(S):
        n = min(int(lengths[s]), pages.shape[1] * page_size)
        if n < 0:
            out[s] = np.nan
            continue
        t = np.arange(max(0, n - window) if window else 0, n)
        p = pages[s][t // page_size] if t.size else np.zeros(0, int)
        ok = (p >= 0) & (p < k.shape[0])
        t, p = t[ok], p[ok]
        if not t.size:
            continue
        for h in range(heads):
            kh = k[p, h // (heads // kv_heads), t % page_size]
            vh = v[p, h // (heads // kv_heads), t % page_size]
            score = kh @ q[s, h] * scale
            e = np.exp(score - score.max())
            w = e / e.sum()
            out[s, h] = w @ vh
            # a score's f32 sum, the maximum's, the exponential and its argument; p in two bf16 parts; the sums over the tokens
            off = 2 * (np.abs(kh) @ np.abs(q[s, h]) * abs(scale)).max() * (dim + 8) * U32
            off += 4 * U32 * np.abs(score - score.max()).max() + 2.0 ** -15 + (n / 16 + 160) * U32
            room[s, h] = (w @ np.abs(vh)) * off
    return out, room
