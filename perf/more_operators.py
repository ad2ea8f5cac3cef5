"""Timed cases of what a decoder layer does between its projections: the RMS norm that adds the residual and rounds for
the next projection, rotary positions, the 8-bit key-value cache (written with its rounding, read back), and the
attention of one new token per sequence over that cache.

Values held in 8 bits are code * scale, with one f32 scale for a token (norm), for 128 inputs of a token (norm, block)
or for a token and head (cache): scale = absmax / 127 (int8) or absmax / 448 (E4M3).  The cache is kept in pages,
[pages, kv_heads, page_size, dim]; slot p * page_size + i is place i of page p.
`run` computes an operator in plain torch operations, or through the framework's entry points where `own` is true.
"""
import math

import torch

own = False

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
MOST = {"int8": 127.0, "fp8": 448.0, "fp8_block": 448.0}


def listed():
    return [
        # one decoded token before q, k and v: residual added, rounded to int8 (the shortest call of a decode step)
        {"name": "norm_decode_int8", "op": "norm", "M": 1, "K": 4096, "out": "int8", "residual": True},
        # a ragged batch of odd width before block-scaled E4M3 products
        {"name": "norm_odd_block", "op": "norm", "M": 333, "K": 1408, "out": "fp8_block", "residual": True},
        # a batch of long prompts, rounded to E4M3 by the token
        {"name": "norm_prompt_fp8", "op": "norm", "M": 8192, "K": 4096, "out": "fp8", "residual": True},
        # interleaved pairs in half of short heads, an odd number of heads and tokens, positions stretched evenly
        {"name": "rope_odd_interleaved", "op": "rope", "T": 333, "heads": 13, "dim": 64, "dims": 32, "interleaved": True, "norm": False,
         "base": 10000.0, "scaling": "linear", "factor": 4.0, "original": 4096},
        # the queries of a long prompt, each head normalised first, frequencies of a context four times the trained one
        {"name": "rope_prompt_norm", "op": "rope", "T": 4096, "heads": 32, "dim": 128, "dims": 128, "interleaved": False, "norm": True,
         "base": 1000000.0, "scaling": "yarn", "factor": 4.0, "original": 32768},
        # a decode step of a padded batch: q, k and v of one projection rotated, k and v into an E4M3 cache
        {"name": "write_decode_fp8", "op": "write", "T": 16, "pad": 3, "heads": 32, "kv_heads": 8, "dim": 128, "kind": "fp8", "page": 16,
         "dims": 128, "interleaved": False, "norm": False, "base": 500000.0, "scaling": "bands", "factor": 8.0, "original": 8192},
        # a prompt's keys and values into an int8 cache, and read back as the prompt's own attention takes them
        {"name": "write_prompt_int8", "op": "write", "T": 4096, "pad": 0, "heads": 32, "kv_heads": 8, "dim": 128, "kind": "int8", "page": 64,
         "dims": 128, "interleaved": False, "norm": True, "base": 1000000.0, "scaling": "none", "factor": 1.0, "original": 40960},
        # a short prefix of another request read back from an int8 cache of odd head length
        {"name": "read_odd_int8", "op": "read", "n": 517, "kv_heads": 5, "dim": 80, "kind": "int8", "page": 48},
        # long prefixes read back from an E4M3 cache
        {"name": "read_long_fp8", "op": "read", "n": 65536, "kv_heads": 8, "dim": 128, "kind": "fp8", "page": 64},
        # one sequence of an ordinary length, alone
        {"name": "attn_one_int8", "op": "attn", "S": 1, "heads": 32, "kv_heads": 8, "dim": 128, "kind": "int8", "page": 16, "shortest": 777,
         "longest": 777, "empty": 0, "pad": 0, "window": 0},
        # a ragged, padded batch over an unrounded cache: five queries to a key head, a window, a sequence without tokens
        {"name": "attn_ragged_bf16", "op": "attn", "S": 37, "heads": 20, "kv_heads": 4, "dim": 64, "kind": "bf16", "page": 48, "shortest": 1,
         "longest": 5000, "empty": 1, "pad": 2, "window": 2048},
        # long contexts: the cache of a layer past what the caches of the chip hold
        {"name": "attn_long_fp8", "op": "attn", "S": 8, "heads": 32, "kv_heads": 8, "dim": 128, "kind": "fp8", "page": 64, "shortest": 16000,
         "longest": 32768, "empty": 0, "pad": 0, "window": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "write", "read", "attn", "attn"])
    if op == "norm":
        out = rng.choice(["int8", "fp8", "fp8_block", "bf16"])
        step = 128 if out == "fp8_block" else 16
        K = step * max(1, _log_int(rng, 128, 16384) // step)
        return {"op": op, "M": max(1, _log_int(rng, 1, 8192) * 4096 // max(K, 4096)), "K": K, "out": out, "residual": rng.random() < 0.7}
    dim = rng.choice([64, 80, 96, 128, 128, 256])
    turn = {"dims": rng.choice([dim, dim, 16 * rng.randint(1, dim // 16)]), "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.5,
            "base": rng.choice([10000.0, 500000.0, 1000000.0]), "scaling": rng.choice(["none", "linear", "ntk", "yarn", "bands"]),
            "factor": rng.choice([2.0, 4.0, 8.0]), "original": rng.choice([4096, 8192, 32768])}
    if turn["dims"] == 16 and turn["scaling"] in ("ntk", "yarn"):
        turn["scaling"] = "linear"
    if op == "rope":
        heads = rng.randint(1, 40)
        return {"op": op, "T": _log_int(rng, 1, 4096 * 4096 // (dim * max(heads, 32))), "heads": heads, "dim": dim, **turn}
    kv_heads, kind, page = rng.randint(1, 8), rng.choice(["bf16", "int8", "fp8"]), 16 * rng.randint(1, 8)
    heads = kv_heads * rng.choice([1, 2, 4, 5, 8])
    if op == "write":
        T = _log_int(rng, 1, 2048)
        return {"op": op, "T": T, "pad": rng.randint(0, T // 4), "heads": heads, "kv_heads": kv_heads, "dim": dim, "kind": kind, "page": page, **turn}
    if op == "read":
        return {"op": op, "n": _log_int(rng, 1, 32768 * 128 // dim), "kv_heads": kv_heads, "dim": dim, "kind": kind, "page": page}
    S = _log_int(rng, 1, 64)
    longest = _log_int(rng, 1, min(32768, 8 * 32768 * 128 // (S * max(dim, 128) * (2 if kind == "bf16" else 1))))
    return {"op": op, "S": S, "heads": heads, "kv_heads": kv_heads, "dim": dim, "kind": kind, "page": page, "shortest": rng.randint(1, longest),
            "longest": longest, "empty": rng.randint(0, S // 8), "pad": rng.randint(0, S // 8), "window": rng.choice([0, 0, _log_int(rng, 16, 8192)])}


# ---- inputs ---------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, M, K):
    """bf16 activations: N(0, 1) with 8 channels 20 times larger, as layer inputs have them."""
    x = _normal(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[:8]] *= 20.0
    return x.to(BF16)


def _lengths(case):
    """Tokens of each sequence: spread between the shortest and the longest, the empty ones, then rows that hold none."""
    live = case["S"] - case["empty"] - case["pad"]
    spread = case["longest"] - case["shortest"]
    lengths = [case["longest"] - int(spread * (i * 0.6180339887 % 1.0)) for i in range(live)]
    return lengths + [0] * case["empty"] + [-1] * case["pad"]


def _cache(g, case, pages):
    """The cache's tensors, holding earlier tokens of other requests."""
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    c = {"kind": case["kind"], "page": case["page"]}
    for n in ("k", "v"):
        x = _normal(g, *shape)
        if n == "k":   # a few channels of the keys are larger than the others
            x[..., torch.randperm(case["dim"], generator=g, device="cuda")[:2]] *= 4.0
        if case["kind"] == "bf16":
            c[n], c[n + "_scale"] = x.to(BF16), None
        else:
            c[n] = (x * 32).clamp_(-127, 127).round_().to(torch.int8) if case["kind"] == "int8" else (x * 64).clamp_(-448, 448).to(E4M3)
            c[n + "_scale"] = (torch.rand(shape[:3], generator=g, device="cuda") + 0.5) / (32 if case["kind"] == "int8" else 64)
    return c


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": dict(case)}
    if op == "norm":
        M, K = case["M"], case["K"]
        s["x"], s["gamma"] = _activations(g, M, K), (1 + 0.2 * _normal(g, K)).to(BF16)
        # the residual stream that a pass finds; the sum goes to a tensor of its own, so that every pass finds the same
        s["residual"] = (2 * _normal(g, M, K)).to(BF16) if case["residual"] else None
        if case["out"] == "bf16":
            s["y"] = torch.empty((M, K), dtype=BF16, device="cuda")
        else:
            s["q"] = torch.empty((M, K), dtype=torch.int8 if case["out"] == "int8" else E4M3, device="cuda")
            s["s"] = torch.empty((M, K // 128) if case["out"] == "fp8_block" else (M,), dtype=F32, device="cuda")
        if case["residual"]:
            s["sum"] = torch.empty((M, K), dtype=BF16, device="cuda")
        return s
    if op in ("rope", "write"):
        T, heads, dim = case["T"], case["heads"], case["dim"]
        s["positions"] = torch.randint(0, int(case["original"] * case["factor"]), (T,), generator=g, device="cuda", dtype=torch.int32)
        s["frequencies"], s["strength"] = _frequencies(case)
        s["gammas"] = [(1 + 0.2 * _normal(g, dim)).to(BF16) for _ in range(2)] if case["norm"] else [None, None]
        s["out"] = torch.empty((T, heads, dim), dtype=BF16, device="cuda")
        if own:
            import quantized_linear_layers_token_amd as Q
            s["rope"] = Q.Rope(case["dims"], base=case["base"], scaling=case["scaling"], factor=case["factor"], original=case["original"],
                               interleaved=case["interleaved"], device="cuda")
    if op == "rope":
        s["x"] = (_normal(g, T, heads, dim) * 2).to(BF16)
        return s
    if op == "write":
        wide = case["heads"] + 2 * case["kv_heads"]   # q, k and v as one projection leaves them
        s["qkv"] = (_normal(g, T, wide, dim) * 2).to(BF16)
        pages = -(-T // case["page"]) + 1
        s["slots"] = torch.randperm(pages * case["page"], generator=g, device="cuda")[:T].to(torch.int32)
        s["slots"][T - case["pad"]:] = -1             # rows behind the last sequence
    elif op == "read":
        pages = -(-case["n"] // case["page"]) + 1
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(case["n"], device="cuda")
        s["slots"] = (order[at // case["page"]] * case["page"] + at % case["page"]).to(torch.int32)
    else:
        lengths = _lengths(case)
        wide = -(-max(1, max(lengths)) // case["page"])
        held = [-(-max(0, n) // case["page"]) for n in lengths]
        pages = sum(held) + 1
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["pages"] = torch.zeros((case["S"], wide), dtype=torch.int32, device="cuda")
        first = 0
        for i, n in enumerate(held):
            s["pages"][i, :n] = order[first:first + n]
            first += n
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        s["x"] = (_normal(g, case["S"], case["heads"], case["dim"]) * 1.5).to(BF16)
        s["out"] = torch.full((case["S"], case["heads"], case["dim"]), 0.25, dtype=BF16, device="cuda")
    s["cache"] = _cache(g, case, pages)
    if op == "read" or (op == "write" and case["kind"] == "int8"):
        rows = (s["slots"].numel(), case["kv_heads"], case["dim"])
        s["read"] = [torch.full(rows, 0.5, dtype=BF16, device="cuda") for _ in range(2)]
    if own:
        import quantized_linear_layers_token_amd as Q
        s["kv"] = Q.KVCache(*(s["cache"][n] for n in ("k", "v", "k_scale", "v_scale")))
        if op == "attn":
            s["workspace"] = torch.empty(Q.qlin_attn_decode_workspace(case["heads"], s["kv"]), dtype=torch.uint8, device="cuda")
    return s


# ---- the operators --------------------------------------------------------

def _frequencies(case):
    """(f64 angles per position of each pair, the factor of cosine and sine)."""
    n, base, factor, original = case["dims"], case["base"], case["factor"], case["original"]
    i = torch.arange(0, n, 2, dtype=F64, device="cuda") / n
    if case["scaling"] == "ntk":
        return (base * factor ** (n / (n - 2))) ** -i, 1.0
    f = base ** -i
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "bands":   # turns within the trained length: 4 and more stay, 1 and fewer are stretched
        turns = original * f / (2 * math.pi)
        keep = ((turns - 1) / 3).clamp(0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    if case["scaling"] == "yarn":    # pairs of 32 turns and more stay, of one and fewer are stretched, a ramp over the pairs between
        place = lambda t: n * math.log(original / (t * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(place(32)), 0), min(math.ceil(place(1)), n - 1)
        ramp = ((torch.arange(n // 2, dtype=F64, device="cuda") - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    return f, 1.0


def _rounded(x, kind):
    """(values of the codes before rounding, scales) of x over its last axis, in f32."""
    a = x.abs().amax(-1, keepdim=True)
    inv = torch.where(a > 0, MOST[kind] / a, 0.0)
    return x * inv, (a / MOST[kind]).squeeze(-1)


def _codes(t, kind):
    return t.round().clamp(-127, 127).to(torch.int8) if kind == "int8" else t.clamp(-448, 448).to(E4M3)


def _run_norm(s):
    c, x = s["case"], s["x"].to(F32)
    r = x
    if c["residual"]:
        s["sum"].copy_(x + s["residual"].to(F32))
        r = s["sum"].to(F32)
    size = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6)
    t = r * s["gamma"].to(F32)   # (a product of two bf16 values: exact)
    if c["out"] == "bf16":
        return {"y": (t * size).to(BF16), "sum": s.get("sum")}
    if c["out"] == "fp8_block":
        q, scale = _rounded(t.unflatten(1, (-1, 128)), "fp8")
        return {"q": _codes(q.flatten(1), "fp8"), "s": scale * size, "sum": s.get("sum")}
    q, scale = _rounded(t, c["out"])
    return {"q": _codes(q, c["out"]), "s": scale * size.squeeze(1), "sum": s.get("sum")}


def _turned(x, s, gamma):
    """Heads x [T, H, dim], normalised where gamma is given, their first dims channels rotated, in f32."""
    c, x = s["case"], x.to(F32)
    if gamma is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * gamma.to(F32)
    angle = s["positions"].to(F64).unsqueeze(1) * s["frequencies"]
    cos, sin = ((f(angle) * s["strength"]).to(F32).unsqueeze(1) for f in (torch.cos, torch.sin))
    turn, rest = x[..., :c["dims"]], x[..., c["dims"]:]
    if c["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turn.chunk(2, -1)
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _run_write(s):
    c, cache = s["case"], s["cache"]
    q, k, v = s["qkv"].split((c["heads"], c["kv_heads"], c["kv_heads"]), 1)
    out = {"q": _turned(q, s, s["gammas"][0]).to(BF16)}
    live = s["slots"] >= 0
    slots = s["slots"][live].to(torch.int64)
    page, place = slots // c["page"], slots % c["page"]
    for n, x in (("k", _turned(k, s, s["gammas"][1])), ("v", v.to(F32))):
        if c["kind"] == "bf16":
            cache[n][page, :, place] = x[live].to(BF16)
        else:
            t, scale = _rounded(x[live], c["kind"])
            cache[n].view(torch.int8)[page, :, place] = _codes(t, c["kind"]).view(torch.int8)
            cache[n + "_scale"][page, :, place] = scale
    if c["kind"] != "int8":
        return {**out, **{n: cache[n] for n in ("k", "v", "k_scale", "v_scale")}}
    read = _run_read(s)
    return {**out, "read": read, "k_scale": cache["k_scale"], "v_scale": cache["v_scale"]}


def _run_read(s):
    c, cache = s["case"], s["cache"]
    slots = s["slots"].to(torch.int64)
    page, place = slots.clamp(min=0) // c["page"], slots.clamp(min=0) % c["page"]
    live = (slots >= 0).view(-1, 1, 1)
    rows = []
    for n, was in zip(("k", "v"), s["read"]):
        x = cache[n].view(torch.int8)[page, :, place].view(cache[n].dtype) if c["kind"] == "fp8" else cache[n][page, :, place]
        x = x.to(F32)
        if c["kind"] != "bf16":
            x = x * cache[n + "_scale"][page, :, place].unsqueeze(-1)
        rows.append(torch.where(live, x.to(BF16), was))
    return rows


def _run_attn(s):
    c, cache = s["case"], s["cache"]
    S, group = c["S"], c["heads"] // c["kv_heads"]
    held = []
    for n in ("k", "v"):
        t = cache[n].view(torch.int8)[s["pages"]].view(cache[n].dtype) if c["kind"] == "fp8" else cache[n][s["pages"]]
        x = t.to(F32)                                            # [S, pages, kv_heads, page, dim]
        if c["kind"] != "bf16":
            x = x * cache[n + "_scale"][s["pages"]].unsqueeze(-1)
        held.append(x.transpose(1, 2).flatten(2, 3).flatten(0, 1))   # [S * kv_heads, tokens, dim]
    k, v = held
    q = s["x"].to(F32).view(S * c["kv_heads"], group, c["dim"])
    scores = torch.bmm(k, q.transpose(1, 2).contiguous()).transpose(1, 2) / math.sqrt(c["dim"])
    at, length = torch.arange(k.shape[1], device="cuda"), s["lengths"].unsqueeze(1)
    live = at < length
    if c["window"]:
        live = live & (at >= length - c["window"])
    live = live.repeat_interleave(c["kv_heads"], 0).unsqueeze(1)
    scores = torch.where(live, scores, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    sums = e.sum(-1, keepdim=True)
    p = torch.where(sums > 0, e / torch.where(sums > 0, sums, 1.0), 0.0)
    y = torch.bmm(p, v).view(S, c["heads"], c["dim"]).to(BF16)
    return torch.where((s["lengths"] < 0).view(-1, 1, 1), s["out"], y)


def run(s):
    op, c = s["case"]["op"], s["case"]
    if not own:
        return {"norm": _run_norm, "rope": lambda t: _turned(t["x"], t, t["gammas"][0]).to(BF16), "write": _run_write, "read": _run_read,
                "attn": _run_attn}[op](s)
    import quantized_linear_layers_token_amd as Q
    if op == "norm":
        if c["out"] == "bf16":
            Q.qlin_norm_bf16(s["x"], s["gamma"], s["y"], residual=s["residual"], sum_out=s.get("sum"), eps=1e-6)
            return {"y": s["y"], "sum": s.get("sum")}
        if c["out"] == "int8":
            Q.qlin_norm_int8(s["x"], s["gamma"], s["q"], s["s"], residual=s["residual"], sum_out=s.get("sum"), eps=1e-6)
        else:
            Q.qlin_norm_fp8(s["x"], s["gamma"], s["q"], s["s"], group=128 if c["out"] == "fp8_block" else 0, residual=s["residual"],
                            sum_out=s.get("sum"), eps=1e-6)
        return {"q": s["q"], "s": s["s"], "sum": s.get("sum")}
    if op == "rope":
        Q.qlin_rope(s["x"], s["positions"], s["rope"], s["out"], gamma=s["gammas"][0], eps=1e-6)
        return s["out"]
    if op == "write":
        q, k, v = s["qkv"].split((c["heads"], c["kv_heads"], c["kv_heads"]), 1)
        Q.qlin_cache_write(s["kv"], s["slots"], k, v, positions=s["positions"], rope=s["rope"], q=q, q_out=s["out"], q_gamma=s["gammas"][0],
                           k_gamma=s["gammas"][1], eps=1e-6)
        if c["kind"] != "int8":
            return {"q": s["out"], **{n: s["cache"][n] for n in ("k", "v", "k_scale", "v_scale")}}
        Q.qlin_cache_read(s["kv"], s["slots"], *s["read"])
        return {"q": s["out"], "read": s["read"], "k_scale": s["cache"]["k_scale"], "v_scale": s["cache"]["v_scale"]}
    if op == "read":
        Q.qlin_cache_read(s["kv"], s["slots"], *s["read"])
        return s["read"]
    Q.qlin_attn_decode(s["x"], s["kv"], s["pages"], s["lengths"], s["out"], s["workspace"], window=c["window"])
    return s["out"]


# ---- what they cannot do without ------------------------------------------

def _row_bytes(case):
    """Bytes of a token's keys (or values) in the cache, scales among them."""
    return case["kv_heads"] * (2 * case["dim"] if case["kind"] == "bf16" else case["dim"] + 4)


def work(case):
    op = case["op"]
    if op == "norm":
        M, K = case["M"], case["K"]
        out = 2 * K if case["out"] == "bf16" else K + 4 * (K // 128 if case["out"] == "fp8_block" else 1)
        return {"bytes": M * (2 * K + (4 * K if case["residual"] else 0) + out) + 2 * K, "flops": 6 * M * K}
    if op == "rope":
        n = case["T"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["T"], "flops": 6 * n}
    if op == "write":
        T, live, dim = case["T"], case["T"] - case["pad"], case["dim"]
        n = T * case["heads"] * dim
        b = 4 * n + 8 * T + live * (4 * case["kv_heads"] * dim + 2 * _row_bytes(case))
        if case["kind"] == "int8":   # read back
            b += live * (2 * _row_bytes(case) + 4 * case["kv_heads"] * dim)
        return {"bytes": b, "flops": 6 * (n + 2 * live * case["kv_heads"] * dim)}
    if op == "read":
        return {"bytes": case["n"] * (2 * _row_bytes(case) + 4 * case["kv_heads"] * case["dim"] + 4), "flops": 2 * case["n"] * case["kv_heads"] * case["dim"]}
    tokens = sum(min(max(0, n), case["window"] or n) for n in _lengths(case))
    rows = (case["S"] - case["pad"]) * case["heads"] * case["dim"]
    return {"bytes": tokens * 2 * _row_bytes(case) + 4 * rows + 4 * case["S"], "flops": 4 * tokens * case["heads"] * case["dim"]}


# ---- the definitions in 64 bits -------------------------------------------

def _exact_turn(x, s, gamma):
    """Each pair of channels as a complex number times strength * e^(i angle)."""
    c, x = s["case"], x.to(F64)
    if gamma is not None:
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * gamma.to(F64)
    half = c["dims"] // 2
    first = torch.arange(half, device=x.device) * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)
    z = torch.complex(x[..., first], x[..., second])
    angle = torch.outer(s["positions"].to(F64), s["frequencies"])
    z = z * torch.polar(torch.full_like(angle, s["strength"]), angle).unsqueeze(1)
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(cache, n, page, place):
    codes = cache[n].to(F64)[page, :, place] if cache[n].dtype != E4M3 else cache[n].to(F32)[page, :, place].to(F64)
    return codes if cache[n + "_scale"] is None else codes * cache[n + "_scale"].to(F64)[page, :, place].unsqueeze(-1)


def _exact_attn(s):
    c, cache = s["case"], s["cache"]
    y = s["out"].to(F64)
    group = c["heads"] // c["kv_heads"]
    for i, n in enumerate(s["lengths"].tolist()):
        if n < 0:
            continue
        y[i] = 0
        at = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device=y.device)
        if not at.numel():
            continue
        page, place = s["pages"][i].to(torch.int64)[at // c["page"]], at % c["page"]
        for h in range(c["kv_heads"]):
            row = {}
            for m in ("k", "v"):
                codes = cache[m][:, h].view(torch.int8)[page, place].view(E4M3).to(F32).to(F64) if c["kind"] == "fp8" else cache[m][page, h, place].to(F64)
                row[m] = codes if cache[m + "_scale"] is None else codes * cache[m + "_scale"][page, h, place].to(F64).unsqueeze(1)
            heads = slice(h * group, (h + 1) * group)
            p = torch.softmax(torch.matmul(s["x"][i, heads].to(F64), row["k"].t()) / math.sqrt(c["dim"]), 1)
            y[i, heads] = torch.matmul(p, row["v"])
    return y


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    c = s["case"]
    if op == "norm":
        x, total = s["x"].to(F64), None
        if c["residual"]:
            total = x + s["residual"].to(F64)
            x = total.to(F32).to(BF16).to(F64)   # the residual stream is bf16, and its norm is taken
        y = x * s["gamma"].to(F64) / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()
        if c["out"] == "bf16":
            return {"y": y, "sum": total}
        rows = y.unflatten(1, (-1, 128)) if c["out"] == "fp8_block" else y.unsqueeze(1)
        a = rows.abs().amax(2)
        scale = a / MOST[c["out"]]
        codes = None if c["out"] == "int8" else (rows / scale.unsqueeze(2)).flatten(1)
        return {"q": codes, "s": scale if c["out"] == "fp8_block" else scale.squeeze(1), "sum": total}
    if op == "rope":
        return _exact_turn(s["x"], s, s["gammas"][0])
    cache = s.get("cache")
    if op == "write":
        heads, kv = c["heads"], c["kv_heads"]
        out = {"q": _exact_turn(s["qkv"][:, :heads], s, s["gammas"][0])}
        rows = {"k": _exact_turn(s["qkv"][:, heads:heads + kv], s, s["gammas"][1]), "v": s["qkv"][:, heads + kv:].to(F64)}
        held, back = {}, []
        live = torch.nonzero(s["slots"] >= 0).flatten()
        page, place = (f(s["slots"][live].to(torch.int64), c["page"]) for f in (torch.div, torch.remainder))
        page = page.floor().to(torch.int64)
        for n in ("k", "v"):
            values = cache[n].to(F32).to(F64)
            scale = None if cache[n + "_scale"] is None else cache[n + "_scale"].to(F64)
            x = rows[n][live]
            if scale is not None:
                a = x.abs().amax(-1) / MOST[c["kind"]]
                scale[page, :, place] = a
                values[page, :, place] = x / a.unsqueeze(-1)
                if c["kind"] == "int8":   # (whole numbers: what is read back is a rounded one times its scale)
                    x = values[page, :, place].round() * a.unsqueeze(-1)
            else:
                values[page, :, place] = x
            held[n], held[n + "_scale"] = values, scale
            whole = torch.full(rows[n].shape, 0.5, dtype=F64, device=x.device)
            whole[live] = x
            back.append(whole)
        if c["kind"] != "int8":
            return {**out, **held}
        return {**out, "read": back, "k_scale": held["k_scale"], "v_scale": held["v_scale"]}
    if op == "read":
        slots = s["slots"].to(torch.int64)
        return [_exact_rows(cache, n, slots // c["page"], slots % c["page"]) for n in ("k", "v")]
    return _exact_attn(s)
