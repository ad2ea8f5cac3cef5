"""The router's definition in 64 bits, masked experts and groups included (NumPy, independent of the library)."""
import numpy as np

BIG = np.finfo(np.float64).max
LARGEST = np.float64(np.finfo(np.float32).max)


def finite(v):
    """NaN and minus infinity count as the smallest value, infinity as the largest."""
    return -BIG if np.isnan(v) else float(min(max(v, -BIG), BIG))


def route_token(logits, k, score, bias, groups, top_groups, group_best, renorm, scale):
    """One token: -> (ids, weights).  A masked expert (logit minus infinity or NaN) has score 0, counts for no run's
    worth and comes after every live expert of the runs that stay; a run without a live expert comes after the others."""
    E = len(logits)
    live = [bool(v > -np.inf) for v in logits]
    l = [min(float(v), LARGEST) if on else None for v, on in zip(logits, live)]
    if score == 0:
        m = max((v for v in l if v is not None), default=0.0)
        e = [np.exp(v - m) if v is not None else 0.0 for v in l]
        total = sum(e)
        s = [v / total if total else 0.0 for v in e]
    else:
        with np.errstate(over="ignore"):
            s = [1.0 / (1.0 + np.exp(-v)) if v is not None else 0.0 for v in l]
    if bias is None and (groups == 1 or group_best == 1):   # the order of the choices is that of the logits
        choice = l
    else:
        with np.errstate(invalid="ignore", over="ignore"):
            choice = [finite(s[e] + (0.0 if bias is None else float(bias[e]))) if live[e] else None for e in range(E)]
    size = E // groups
    runs = []
    for g in range(groups):
        best = sorted((choice[e] for e in range(g * size, (g + 1) * size) if live[e]), reverse=True)[:group_best]
        with np.errstate(over="ignore"):
            runs.append((not best, -finite(np.float64(sum(np.float64(v) for v in best))), g))
    stay = [g for _, _, g in sorted(runs)[:top_groups]]
    allowed = [e for g in sorted(stay) for e in range(g * size, (g + 1) * size)]
    ids = sorted(allowed, key=lambda e: (not live[e], -choice[e] if live[e] else 0.0, e))[:k]
    w = np.array([s[e] for e in ids])
    if renorm:
        w = w / w.sum() if w.sum() > 0 else np.zeros(k)
    return ids, w * scale


def route(logits, k, score=0, bias=None, groups=1, top_groups=1, group_best=2, renormalize=True, scale=1.0):
    """logits f32 [T, E] -> (ids [T, k], weights in 64 bits [T, k])."""
    rows = [route_token(row, k, score, bias, groups, top_groups, group_best, renormalize, scale) for row in logits]
    return np.array([r[0] for r in rows]), np.array([r[1] for r in rows])
