"""Decode steps of a layer's attention half, as a program runs them: norm with residual -> q, k and v -> rotation and cache ->
attention -> output projection -> norm with residual, on W8A8 and block FP8 projections.  Every stage is checked from what
the one before it gave; the whole step is captured too, and its replays equal the eager steps bit for bit."""
import numpy as np
import pytest

import layer_reference as R
import oracle as O
import workloads as W
from gpu_helpers import assert_within_tol, dev, host, torch_mod
from test_heads_gpu import contents, within
from test_norm_gpu import check as check_norm

pytestmark = pytest.mark.gpu
H, HEADS, KV, DIM, PAGE, S = 512, 8, 2, 64, 16, 5


def Q():
    import quantized_linear_layers_token_amd as q
    return q


class Step:
    def __init__(self, scheme, kind):
        torch, q = torch_mod(), Q()
        self.scheme, self.kind = scheme, kind
        rng = np.random.default_rng(31)
        self.lengths = np.array([1, 20, 47, 100, -1], np.int32)          # before a step's token; the last row pads the batch
        pages = 32
        self.table = np.concatenate([rng.permutation(pages).reshape(4, 8), np.zeros((1, 8))]).astype(np.int32)
        n = (HEADS + 2 * KV) * DIM
        self.block = scheme == q.SCHEME_FP8_BLOCK
        w = W.w_int8 if scheme == q.SCHEME_W8A8 else W.w_e4m3
        shape = (lambda a, b: (a // 128, b // 128)) if self.block else (lambda a, b: (a,))
        self.wqkv, self.wo = w(1, n, H), w(2, H, HEADS * DIM)
        self.sqkv, self.so = W.scale_bf16(3, shape(n, H)), W.scale_bf16(4, shape(H, HEADS * DIM))
        self.g1, self.g2, self.qg, self.kg = (R.bits(1 + 0.2 * rng.standard_normal(m)) for m in (H, H, DIM, DIM))
        d = {m: dev(getattr(self, m)) for m in ("wqkv", "wo", "sqkv", "so", "g1", "g2", "qg", "kg", "table")}
        self.d = d
        self.cache = q.KVCache.empty(pages, KV, PAGE, DIM, {"bf16": torch.bfloat16, "int8": torch.int8, "fp8": torch.uint8}[kind])
        for m in ("k", "v"):                                             # what the earlier tokens left
            t = getattr(self.cache, m)
            raw = W.x_bf16(5, 1, t.numel()).reshape(t.shape) if kind == "bf16" else rng.integers(0, 0x60, tuple(t.shape)).astype(np.int8 if kind == "int8" else np.uint8)
            (t.view(torch.int16) if kind == "bf16" else t).copy_(dev(raw))
            if kind != "bf16":
                getattr(self.cache, m + "_scale").fill_(0.02)
        self.rope = q.Rope(DIM, 5e5, "bands", 8.0, 8192)
        e = lambda *shape, dtype=torch.int16: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731
        f32, i32, u8 = torch.float32, torch.int32, torch.uint8
        groups = (lambda k: (S, k // 128)) if self.block else (lambda k: (S,))
        self.t = dict(x=e(S, H), residual=e(S, H), sum=e(S, H), qx=e(S, H, dtype=u8), sx=e(*groups(H), dtype=f32),
                      qkv=e(S, n), q=e(S, HEADS, DIM), attn=e(S, HEADS, DIM), qa=e(S, HEADS * DIM, dtype=u8), sa=e(*groups(HEADS * DIM), dtype=f32),
                      o=e(S, H), sum2=e(S, H), qx2=e(S, H, dtype=u8), sx2=e(*groups(H), dtype=f32), positions=e(S, dtype=i32), slots=e(S, dtype=i32),
                      lengths=e(S, dtype=i32), work=e(q.qlin_attn_decode_workspace(HEADS, self.cache), dtype=u8))

    def norm(self, x, g, qx, sx, residual, total):
        q = Q()
        if self.scheme == q.SCHEME_W8A8:
            q.qlin_norm_int8(x, g, qx, sx, residual=residual, sum_out=total)
        else:
            q.qlin_norm_fp8(x, g, qx, sx, group=128 if self.block else 0, residual=residual, sum_out=total)

    def run(self):
        q, t, d = Q(), self.t, self.d
        self.norm(t["x"], d["g1"], t["qx"], t["sx"], t["residual"], t["sum"])
        gemm = {q.SCHEME_W8A8: q.qlin_gemm_w8a8, q.SCHEME_FP8_ROWWISE: q.qlin_gemm_fp8_rowwise, q.SCHEME_FP8_BLOCK: q.qlin_gemm_fp8_block}[self.scheme]
        gemm(t["qx"], t["sx"], d["wqkv"], d["sqkv"], t["qkv"])
        heads = t["qkv"].view(S, HEADS + 2 * KV, DIM)
        qh, kh, vh = heads.split((HEADS, KV, KV), 1)
        q.qlin_cache_write(self.cache, t["slots"], kh, vh, positions=t["positions"], rope=self.rope, q=qh, q_out=t["q"], q_gamma=d["qg"], k_gamma=d["kg"])
        q.qlin_attn_decode(t["q"], self.cache, d["table"], t["lengths"], t["attn"], t["work"])
        q.qlin_linear(self.scheme, t["attn"].view(S, HEADS * DIM), [(d["wo"], d["so"], t["o"])], q_x=t["qa"], s_x=t["sa"])
        self.norm(t["o"], d["g2"], t["qx2"], t["sx2"], t["sum"], t["sum2"])

    def begin(self, n):
        """The inputs of the n-th step."""
        rng = np.random.default_rng([77, n])
        before = np.where(self.lengths < 0, 0, self.lengths + n)
        slots = np.where(self.lengths < 0, -1, self.table[np.arange(S), before // PAGE] * PAGE + before % PAGE).astype(np.int32)
        new = {"x": R.bits(rng.standard_normal((S, H))), "residual": R.bits(2 * rng.standard_normal((S, H))), "positions": before.astype(np.int32),
               "slots": slots, "lengths": np.where(self.lengths < 0, -1, before + 1).astype(np.int32)}
        for m, v in new.items():
            self.t[m].copy_(dev(v))
        self.now = new

    def check(self):
        q, t, now = Q(), self.t, self.now
        kind = {q.SCHEME_W8A8: "int8", q.SCHEME_FP8_ROWWISE: "fp8", q.SCHEME_FP8_BLOCK: "block"}[self.scheme]
        decode = (lambda c: c.view(np.int8).astype(np.float64)) if kind == "int8" else O.e4m3_decode
        check_norm(kind, now["x"], now["residual"], self.g1, (host(t["sum"]), decode(host(t["qx"])), host(t["sx"])))
        # the product, from its rounded inputs
        qx, sx = host(t["qx"]), host(t["sx"])
        if kind == "int8":
            y = O.rescale_rowwise(O.contract_int8(qx.view(np.int8), self.wqkv), sx, self.sqkv)
        elif kind == "fp8":
            y = O.rescale_rowwise(O.contract_e4m3(qx, self.wqkv), sx, self.sqkv)
        else:
            y = O.rescale_block(O.contract_e4m3_blocks(qx, self.wqkv), sx, self.sqkv)
        assert_within_tol(host(t["qkv"]), y, "qkv")
        heads = R.value(host(t["qkv"])).reshape(S, HEADS + 2 * KV, DIM)
        freq = self.rope.frequencies.cpu().numpy()
        ref, slack = R.rotate(heads[:, :HEADS], now["positions"], freq, DIM, False, 1.0, R.value(self.qg))
        within(R.value(host(t["q"])), ref, slack, "queries")
        live = now["slots"] >= 0
        at = (now["slots"][live] // PAGE, now["slots"][live] % PAGE)
        stored = {}
        for m, part, gamma in (("k", heads[:, HEADS:HEADS + KV], self.kg), ("v", heads[:, HEADS + KV:], None)):
            ref, slack = (part, np.zeros_like(part)) if gamma is None else R.rotate(part, now["positions"], freq, DIM, False, 1.0, R.value(gamma))
            values, _, s = contents(self.cache, self.kind, m)
            stored[m] = (values if s is None else values * s.astype(np.float64)[..., None]).swapaxes(1, 2)
            got = stored[m].swapaxes(1, 2)[at]
            # half a step: of bf16, of the head's absmax / 127, of E4M3 (2^-4, or of its smallest step)
            a = np.abs(ref[live]).max(-1, keepdims=True)
            half = {"bf16": np.abs(ref[live]) * R.HALF, "int8": a / 127 / 2, "fp8": np.maximum(np.abs(ref[live]) / 16, a / 448 * 2.0 ** -10)}[self.kind]
            assert (np.abs(got - ref[live]) <= half * 1.01 + 2 * slack[live] + a * 8 * R.U32).all(), m
        scale = float(np.float32(DIM ** -0.5))
        ref, room = R.attention(R.value(host(t["q"])), stored["k"], stored["v"], self.table, now["lengths"], PAGE, 0, scale)
        out = R.value(host(t["attn"]))
        assert (out[~live] == 0).all()           # the row that pads the batch, as it was made
        assert (np.abs(out - ref)[live] <= (np.abs(ref) * R.HALF + room * (1 + R.HALF))[live]).all()
        flat = host(t["attn"]).view(np.uint16).reshape(S, -1)
        linear = {"int8": O.linear_w8a8, "fp8": O.linear_fp8_rowwise, "block": O.linear_fp8_block}[kind]
        assert_within_tol(host(t["o"]), linear(flat, self.wo, self.so)[1], "o")
        check_norm(kind, host(t["o"]).view(np.uint16), host(t["sum"]).view(np.uint16), self.g2, (host(t["sum2"]), decode(host(t["qx2"])), host(t["sx2"])))

    def state(self):
        return [v.clone() for v in self.t.values() if v is not self.t["work"]] + [t.clone() for t in (self.cache.k, self.cache.v, self.cache.k_scale, self.cache.v_scale)
                                                                                   if t is not None]


@pytest.mark.parametrize("scheme,kind", [(0, "int8"), (1, "fp8"), (2, "fp8"), (0, "bf16")])
def test_decode_steps(scheme, kind):
    torch = torch_mod()
    eager, replayed = Step(scheme, kind), Step(scheme, kind)
    replayed.begin(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        replayed.run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.run()
    for n in range(4):
        print(f"scheme {scheme}, cache {kind}, step {n}", flush=True)
        eager.begin(n)
        eager.run()
        torch.cuda.synchronize()
        eager.check()
        replayed.begin(n)
        replayed.t["work"].fill_(0xEE)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager.state(), replayed.state()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
