"""Timed cases of the 4-bit operators: projections on 4-bit weights with group scales, routing to experts, and the
experts' gated MLP on 4-bit weights.

Weights are 4-bit codes (two to a byte, the even input in the low half), one bf16 scale per `group` inputs of a row
and, where a case says so, one zero point per scale (else 8):  w[n, k] = (code[n, k] - zero[n, k / group]) * scale[...].
`run` computes an operator in plain torch operations, or through the framework's entry points where `own` is true.
"""
import math

import numpy as np
import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # one token through a square attention output projection: the shortest call of a decode step
        {"name": "decode_o", "op": "linear", "M": 1, "widths": "4096", "K": 4096, "group": 128, "zeros": False, "out": "bf16"},
        # one token through q, k and v with zero points, one call
        {"name": "decode_qkv_zeros", "op": "linear", "M": 1, "widths": "4096,1024,1024", "K": 4096, "group": 64, "zeros": True, "out": "bf16"},
        # one token through the gate/up pair of a large MLP, SwiGLU on the way out
        {"name": "decode_gate_up", "op": "swiglu", "M": 1, "widths": "14336", "K": 4096, "group": 128, "zeros": False, "out": "bf16"},
        # a small ragged batch of decoding sequences through a long-row down projection, f32 results
        {"name": "batch_down_f32", "op": "linear", "M": 13, "widths": "4096", "K": 14336, "group": 128, "zeros": False, "out": "f32"},
        # a prompt of odd length with odd widths, the smallest groups and zero points
        {"name": "prompt_odd", "op": "linear", "M": 333, "widths": "1000,488", "K": 2080, "group": 32, "zeros": True, "out": "bf16"},
        # a long prompt through the down projection: the largest product
        {"name": "prompt_down", "op": "linear", "M": 2048, "widths": "4096", "K": 14336, "group": 128, "zeros": False, "out": "bf16"},
        # routing of one decoded token
        {"name": "route_decode", "op": "route", "T": 1, "E": 128, "k": 8, "score": "softmax", "bias": False, "groups": 1, "top_groups": 1,
         "renorm": True, "scale": 1.0, "logits": "bf16"},
        # routing of a ragged batch over an odd number of experts, weights left as the softmax gives them
        {"name": "route_odd", "op": "route", "T": 333, "E": 60, "k": 4, "score": "softmax", "bias": False, "groups": 1, "top_groups": 1,
         "renorm": False, "scale": 1.0, "logits": "f32"},
        # routing of a long prompt: sigmoid scores, a balancing bias, the best 4 of 8 groups
        {"name": "route_prompt_groups", "op": "route", "T": 4096, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "renorm": True, "scale": 2.5, "logits": "f32"},
        # one decoded token through its experts
        {"name": "experts_decode", "op": "experts", "T": 1, "E": 64, "k": 8, "H": 2048, "I": 1024, "group": 128, "zeros": False, "pad": 0},
        # a padded batch of decoding sequences over odd sizes, a few rows for each expert
        {"name": "experts_batch_odd", "op": "experts", "T": 37, "E": 40, "k": 6, "H": 2048, "I": 736, "group": 32, "zeros": True, "pad": 3},
        # a long prompt through the experts
        {"name": "experts_prompt", "op": "experts", "T": 2048, "E": 64, "k": 8, "H": 2048, "I": 1024, "group": 128, "zeros": False, "pad": 0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "swiglu", "route", "experts"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(max(2, -(-8 // groups)), 512 // groups)
        top_groups = rng.randint(1, groups)
        return {"op": op, "T": _log_int(rng, 1, 8192), "E": E, "k": rng.randint(1, min(16, top_groups * (E // groups))),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
                "renorm": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]), "logits": rng.choice(["bf16", "f32"])}
    group, zeros = rng.choice([32, 64, 128]), rng.random() < 0.5
    if op == "experts":
        E = rng.randint(2, 64)
        return {"op": op, "T": _log_int(rng, 1, 2048), "E": E, "k": rng.randint(1, min(8, E)), "H": group * rng.randint(128 // group, 2048 // group),
                "I": group * rng.randint(128 // group, 1024 // group), "group": group, "zeros": zeros, "pad": 0}
    M = _log_int(rng, 1, 2048)
    K = group * max(1, _log_int(rng, 128, 14336) // group)
    widths = [_log_int(rng, 16, 8192) for _ in range(rng.randint(1, 3) if op == "linear" else 1)]
    if op == "swiglu":
        widths = [8 * max(2, widths[0] // 8)]
    most = 2048 * 4096 * 14336 // (M * K * (2 if op == "swiglu" else 1))
    while sum(widths) > most:
        widths = [max(8, w // 2 // 8 * 8) for w in widths]
    return {"op": op, "M": M, "widths": ",".join(map(str, widths)), "K": K, "group": group, "zeros": zeros,
            "out": rng.choice(["bf16", "f32"]) if op == "linear" else "bf16"}


# ---- inputs ---------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, M, K):
    """bf16 activations: N(0, 1) with 8 channels 20 times larger, as layer inputs have them."""
    x = torch.randn((M, K), generator=g, device="cuda")
    x[:, torch.randperm(K, generator=g, device="cuda")[:8]] *= 20.0
    return x.to(BF16)


def _weights(g, shape, K, group, zeros):
    """Codes [..., N, K/2], scales [..., N, K/group] and zero points (or None)."""
    w = {"codes": torch.randint(0, 256, (*shape, K // 2), dtype=torch.uint8, generator=g, device="cuda"),
         "scales": (torch.rand((*shape, K // group), generator=g, device="cuda") * 4e-3 + 1e-3).to(BF16), "zeros": None}
    if zeros:
        w["zeros"] = torch.randint(5, 11, (*shape, K // group), dtype=torch.uint8, generator=g, device="cuda")
    return w


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": dict(case)}
    if op == "route":
        T, E = case["T"], case["E"]
        # experts differ in how often they are wanted; the bias of a balanced router is small beside the scores
        logits = torch.randn((T, E), generator=g, device="cuda") * 1.5 + 0.5 * torch.randn((E,), generator=g, device="cuda")
        s["logits"] = logits.to(BF16) if case["logits"] == "bf16" else logits
        s["bias"] = 0.1 * torch.randn((E,), generator=g, device="cuda") if case["bias"] else None
        s["ids"] = torch.empty((T, case["k"]), dtype=torch.int32, device="cuda")
        s["weights"] = torch.empty((T, case["k"]), dtype=F32, device="cuda")
        return s
    K, group, zeros = case.get("K"), case["group"], case["zeros"]
    if op == "experts":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        s["x"] = _activations(g, T, H)
        wanted = torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn((E,), generator=g, device="cuda")
        top = torch.topk(wanted, k, dim=1)
        s["ids"] = top.indices.to(torch.int32)
        s["weights"] = torch.softmax(top.values, dim=1)
        if case["pad"]:   # rows behind the batch's last sequence: no expert
            s["ids"][T - case["pad"]:] = -1
        s["w"] = [_weights(g, (E, I), H, group, zeros), _weights(g, (E, I), H, group, zeros), _weights(g, (E, H), I, group, zeros)]
        s["y"] = torch.empty((T, H), dtype=BF16, device="cuda")
    else:
        widths = [int(v) for v in case["widths"].split(",")]
        if op == "swiglu":
            widths *= 2
        s["x"] = _activations(g, case["M"], K)
        s["w"] = [_weights(g, (n,), K, group, zeros) for n in widths]
        out = F32 if case["out"] == "f32" else BF16
        s["y"] = [torch.empty((case["M"], n), dtype=out, device="cuda") for n in (widths[:1] if op == "swiglu" else widths)]
    if own:   # the weights as a program of the framework keeps them, laid out when the model is loaded
        import quantized_linear_layers_token_amd as Q
        s["packed"] = [Q.qlin_pack_w4(w["codes"], w["scales"], w["zeros"]) for w in s["w"]]
        if op == "experts":
            s["workspace"] = torch.empty(Q.qlin_experts_w4_workspace(T, k, *s["packed"]), dtype=torch.uint8, device="cuda")
    return s


# ---- the operators --------------------------------------------------------

def _dequantized(w, index=None):
    """f32 weights [..., N, K] of the codes (of the experts `index` alone, where it is given)."""
    codes, scales, zeros = (t if t is None or index is None else t[index] for t in (w["codes"], w["scales"], w["zeros"]))
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).to(F32)
    q = q.unflatten(-1, (scales.shape[-1], -1))
    q = q - (8.0 if zeros is None else zeros.to(F32).unsqueeze(-1))
    return (q * scales.to(F32).unsqueeze(-1)).flatten(-2)


def _silu(t):
    return t / (1 + torch.exp(-t))


def _run_linear(s):
    x = s["x"].to(F32)
    return [(x @ _dequantized(w).t()).to(y.dtype) for w, y in zip(s["w"], s["y"])]


def _run_swiglu(s):
    x = s["x"].to(F32)
    g, u = (x @ _dequantized(w).t() for w in s["w"])
    return (_silu(g) * u).to(BF16)


def _run_route(s):
    c, logits = s["case"], s["logits"].to(torch.float64)   # 64 bits: scores next to each other decide the choice
    if c["score"] == "softmax":
        e = torch.exp(logits - logits.amax(1, keepdim=True))
        scores = e / e.sum(1, keepdim=True)
    else:
        scores = 1 / (1 + torch.exp(-logits))
    choice = scores if s["bias"] is None else scores + s["bias"].to(torch.float64)
    if c["groups"] > 1:
        by_group = choice.unflatten(1, (c["groups"], -1))
        best = torch.sort(by_group, dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(mask.unsqueeze(2), by_group, -math.inf).flatten(1)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :c["k"]]
    weights = torch.gather(scores, 1, ids)
    if c["renorm"]:
        weights = weights / weights.sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (weights * c["scale"]).to(F32)}


def _run_experts(s):
    c, x, ids, E, T, k = s["case"], s["x"].to(F32), s["ids"].to(torch.int64), s["case"]["E"], s["case"]["T"], s["case"]["k"]
    flat = ids.reshape(-1)
    live = flat >= 0
    if T * k <= E:   # few rows: each with its own expert's weights
        experts = flat.clamp(min=0)
        rows = x.repeat_interleave(k, 0).unsqueeze(2)
        g, u = (torch.bmm(_dequantized(s["w"][i], experts), rows) for i in (0, 1))
        out = torch.bmm(_dequantized(s["w"][2], experts), _silu(g) * u).squeeze(2)
    else:            # rows in the order of their experts, in one batch padded to the fullest expert
        order = torch.sort(torch.where(live, flat, E), stable=True).indices
        counts = torch.bincount(torch.where(live, flat, E), minlength=E + 1)
        expert = torch.where(live, flat, E)[order]
        place = torch.arange(T * k, device="cuda") - (torch.cumsum(counts, 0) - counts)[expert]
        fullest = int(counts.max())
        rows = torch.zeros((E + 1, fullest, c["H"]), device="cuda")
        rows[expert, place] = x[order // k]
        g, u = (torch.bmm(rows[:E], _dequantized(s["w"][i]).transpose(1, 2).contiguous()) for i in (0, 1))
        y = torch.bmm(_silu(g) * u, _dequantized(s["w"][2]).transpose(1, 2).contiguous())
        out = torch.empty((T * k, c["H"]), device="cuda")
        out[order] = y[expert.clamp(max=E - 1), place]
    out = torch.where(live.unsqueeze(1), out * s["weights"].reshape(-1, 1), 0.0)
    return out.unflatten(0, (T, k)).sum(1).to(BF16)


def run(s):
    op, c = s["case"]["op"], s["case"]
    if own:
        import quantized_linear_layers_token_amd as Q
        if op == "linear":
            Q.qlin_linear_w4(s["x"], list(zip(s["packed"], s["y"])), out=Q.OUT_F32 if c["out"] == "f32" else Q.OUT_BF16)
            return s["y"]
        if op == "swiglu":
            Q.qlin_linear_swiglu_w4(s["x"], *s["packed"], s["y"][0])
            return s["y"][0]
        if op == "route":
            Q.qlin_route(s["logits"], s["ids"], s["weights"], score=Q.SCORE_SOFTMAX if c["score"] == "softmax" else Q.SCORE_SIGMOID,
                         bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"])
            return {"ids": s["ids"], "weights": s["weights"]}
        Q.qlin_experts_w4(s["x"], s["ids"], s["weights"], *s["packed"], s["y"], s["workspace"])
        return s["y"]
    return {"linear": _run_linear, "swiglu": _run_swiglu, "route": _run_route, "experts": _run_experts}[op](s)


# ---- what they cannot do without ------------------------------------------

def _weight_bytes(rows, K, group, zeros):
    return rows * K / 2 + rows * (K // group) * (3 if zeros else 2)


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["logits"] == "bf16" else 4
        return {"bytes": T * E * size + T * k * 8 + (4 * E if case["bias"] else 0), "flops": T * E * 4}
    if op == "experts":
        T, E, k, H, I = ((case["T"] - case["pad"]) if n == "T" else case[n] for n in ("T", "E", "k", "H", "I"))
        used = E * (1 - (1 - k / E) ** T)   # the experts that at least one token is expected to want
        return {"bytes": used * (2 * _weight_bytes(I, H, case["group"], case["zeros"]) + _weight_bytes(H, I, case["group"], case["zeros"]))
                + 4 * T * H + 8 * T * k, "flops": 6 * T * k * H * I}
    M, K = case["M"], case["K"]
    widths = [int(v) for v in case["widths"].split(",")]
    rows = sum(widths) * (2 if op == "swiglu" else 1)
    return {"bytes": _weight_bytes(rows, K, case["group"], case["zeros"]) + 2 * M * K + M * sum(widths) * (4 if case["out"] == "f32" else 2),
            "flops": 2 * M * rows * K}


# ---- the definitions in 64 bits -------------------------------------------

def _exact_weight(w, e=None):
    """The weight matrix in 64 bits, from its bytes: low halves are the even inputs, high halves the odd ones."""
    codes, scales = (w["codes"], w["scales"]) if e is None else (w["codes"][e], w["scales"][e])
    zero = 8 if w["zeros"] is None else (w["zeros"] if e is None else w["zeros"][e]).to(torch.float64)
    n, half = codes.shape
    value = torch.empty((n, 2 * half), dtype=torch.float64, device=codes.device)
    value[:, 0::2], value[:, 1::2] = codes % 16, codes // 16
    group = 2 * half // scales.shape[1]
    of = torch.arange(2 * half, device=codes.device) // group
    return (value - (zero if isinstance(zero, int) else zero[:, of])) * scales.to(torch.float64)[:, of]


def _exact_route(s):
    c = s["case"]
    logits = s["logits"].to(torch.float64).cpu().numpy()
    T, E = logits.shape
    if c["score"] == "softmax":
        shifted = np.exp(logits - logits.max(1)[:, None])
        scores = shifted / shifted.sum(1)[:, None]
    else:
        scores = 1.0 / (1.0 + np.exp(-logits))
    choice = scores + (0.0 if s["bias"] is None else s["bias"].cpu().numpy().astype(np.float64))
    ids = np.empty((T, c["k"]), np.int32)
    size = E // c["groups"]
    for t in range(T):
        allowed = list(range(E))
        if c["groups"] > 1:
            worth = [sum(sorted(choice[t, g * size:(g + 1) * size])[-2:]) for g in range(c["groups"])]
            best = sorted(range(c["groups"]), key=lambda g: (-worth[g], g))[:c["top_groups"]]
            allowed = [e for g in best for e in range(g * size, (g + 1) * size)]
        ids[t] = sorted(allowed, key=lambda e: (-choice[t, e], e))[:c["k"]]
    weights = np.take_along_axis(scores, ids.astype(np.int64), 1)
    if c["renorm"]:
        weights = weights / weights.sum(1)[:, None]
    return {"ids": ids, "weights": weights * c["scale"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    x = s["x"].to(torch.float64)
    if case["op"] == "linear":
        return [torch.matmul(x, _exact_weight(w).t()) for w in s["w"]]
    if case["op"] == "swiglu":
        g, u = (torch.matmul(x, _exact_weight(w).t()) for w in s["w"])
        return g * torch.sigmoid(g) * u
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        token, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if token.numel():
            g, u = (torch.matmul(x[token], _exact_weight(w, e).t()) for w in s["w"][:2])
            out = torch.matmul(g * torch.sigmoid(g) * u, _exact_weight(s["w"][2], e).t())
            y.index_add_(0, token, out * s["weights"][token, slot].to(torch.float64).unsqueeze(1))
    return y
