"""Inputs and 64-bit definitions of the 4-bit operators for the tests (NumPy, independent of the library)."""
import numpy as np

U = 2.0 ** -24          # half a step of f32, relative
BF16_HALF = 2.0 ** -8   # half a step of bf16, relative


def bf16_bits(a):
    """f64 array -> bf16 bit patterns, round to nearest even."""
    b = np.ascontiguousarray(a, np.float32).view(np.uint32)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.ascontiguousarray(bits).view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def weights(rng, shape, K, group, zeros, exact=False):
    """codes uint8 [.., N, K/2], bf16 scale bits, zero points or None.  exact: scales are powers of two."""
    codes = rng.integers(0, 256, (*shape, K // 2), dtype=np.uint8)
    if exact:
        scales = bf16_bits(2.0 ** rng.integers(-3, 1, (*shape, K // group)))
    else:
        scales = bf16_bits(rng.uniform(1e-3, 5e-3, (*shape, K // group)))
    zp = rng.integers(0, 16, (*shape, K // group), dtype=np.uint8) if zeros else None
    return codes, scales, zp


def dequantize(w):
    """f64 weights [.., N, K], and the magnitudes (code + zero) * scale of the two terms that the kernels subtract."""
    codes, scales, zp = w
    q = np.empty((*codes.shape[:-1], 2 * codes.shape[-1]))
    q[..., 0::2], q[..., 1::2] = codes & 15, codes >> 4
    rep = q.shape[-1] // scales.shape[-1]
    s = np.repeat(bf16_values(scales), rep, -1)
    z = 8.0 if zp is None else np.repeat(zp.astype(np.float64), rep, -1)
    return (q - z) * s, (q + z) * s


def sum_bound(K, group):
    """Roundings of one f32 result, relative to its terms' magnitudes: at most one for each of K products and K
    terms of the zero point, a scaling and an addition for each group, the join of at most 16 partial sums.
    The matrix cores may cut instead of round: two half steps each."""
    return 2 * U * (2 * K + 3 * (K // group) + 32)


def linear(x, w, group):
    """-> (y in 64 bits, bound of an f32 result's error)."""
    v, mag = dequantize(w)
    return x @ v.T, sum_bound(x.shape[1], group) * (np.abs(x) @ mag.T)


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def swiglu(x, gate, up, group):
    """-> (h in 64 bits, bound of the f32 value that is rounded to h): |silu'| < 1.1, and the exponential, the
    quotient and the product of the f32 evaluation are within 16 half steps (exp: 2 ulp of a rounded argument of
    magnitude |g|, which adds |g| U to its relative error)."""
    g, eg = linear(x, gate, group)
    u, eu = linear(x, up, group)
    h = silu(g) * u
    return h, 1.1 * eg * (np.abs(u) + eu) + np.abs(silu(g)) * eu + (16 + 2 * np.abs(g)) * U * np.abs(h) + 1e-30


def experts(x, ids, weights_, gate, up, down, group, h_half=BF16_HALF):
    """-> (y in 64 bits, bound of the f32 value that is rounded to y).  h_half: relative error of h's rounding."""
    E, I, H = gate[0].shape[0], gate[0].shape[1], x.shape[1]
    y, bound = np.zeros_like(x), np.zeros_like(x)
    one = lambda w, e: tuple(None if t is None else t[e] for t in w)  # noqa: E731
    for e in range(E):
        token, slot = np.nonzero(ids == e)
        if not len(token):
            continue
        h, eh = swiglu(x[token], one(gate, e), one(up, e), group)
        eh = eh * (1 + h_half) + h_half * np.abs(h)
        v, mag = dequantize(one(down, e))
        wt = weights_[token, slot][:, None].astype(np.float64)
        np.add.at(y, token, wt * (h @ v.T))
        row = eh @ np.abs(v).T + sum_bound(I, group) * ((np.abs(h) + eh) @ mag.T)
        np.add.at(bound, token, np.abs(wt) * (row + 3 * U * (np.abs(h) @ np.abs(v).T)))
    return y, bound + U * ids.shape[1] * np.abs(y)


def route(logits, k, score, bias, groups, top_groups, group_best, renorm, scale):
    """-> (ids, weights in 64 bits), token by token from the definition."""
    T, E = logits.shape
    ids, weights_ = np.empty((T, k), np.int64), np.empty((T, k))
    big = np.finfo(np.float64).max
    for t in range(T):
        l = logits[t].astype(np.float64)
        out = ~(l > -np.inf)
        l = np.clip(np.where(out, -np.inf, l), -np.inf, np.finfo(np.float32).max)
        with np.errstate(over="ignore", invalid="ignore"):
            if score == 0:
                p = np.where(out, 0.0, np.exp(l - l.max()))
                s = p / p.sum() if p.sum() else p
            else:
                s = np.where(out, 0.0, 1 / (1 + np.exp(-l)))
            by_logit = bias is None and (groups == 1 or group_best == 1)
            c = l.copy() if by_logit else s + (0 if bias is None else bias.astype(np.float64))
        c = np.where(out, -np.inf, np.where(np.isnan(c), -big, np.clip(c, -big, big)))   # masked: after every other
        size = E // groups
        worth = []
        for g in range(groups):
            best = np.sort(c[g * size:(g + 1) * size])[::-1][:group_best]
            with np.errstate(over="ignore"):
                worth.append(max(best.sum(), -big))
        kept = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
        cand = [e for g in kept for e in range(g * size, (g + 1) * size)]
        ids[t] = sorted(cand, key=lambda e: (-c[e], e))[:k]
        w = s[ids[t]]
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        weights_[t] = w * scale
    return ids, weights_
