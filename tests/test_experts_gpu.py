"""The experts' MLP on 4-bit weights against the 64-bit definition, alone and fed by the router."""
import numpy as np
import pytest

import w4_reference as R
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


def Q():
    import quantized_linear_layers_token_amd as q
    return q


def make(seed, T, E, k, H, I, group, zeros, skew=0.0):
    rng = np.random.default_rng([seed, T, E, H, I])
    xb = R.bf16_bits(rng.standard_normal((T, H)) * np.where(np.arange(H) % 61 == 0, 8.0, 1.0))
    wanted = rng.standard_normal((T, E)) + skew * np.linspace(1, 0, E)
    ids = np.argsort(-wanted, 1)[:, :k].astype(np.int32)
    wt = rng.random((T, k)).astype(np.float32)
    ws = [R.weights(rng, (E, I), H, group, zeros), R.weights(rng, (E, I), H, group, zeros), R.weights(rng, (E, H), I, group, zeros)]
    return xb, ids, wt, ws


def run(xb, ids, wt, ws, packed=None):
    torch = torch_mod()
    q = Q()
    T, H = xb.shape
    packed = packed or [q.qlin_pack_w4(dev(w[0]), dev(w[1]), None if w[2] is None else dev(w[2])) for w in ws]
    size = q.qlin_experts_w4_workspace(T, ids.shape[1], *packed)
    work = torch.full((size + 64,), 0xEE, dtype=torch.uint8, device="cuda")     # poisoned: NaN as h or f32
    raw = torch.full((T * H * 2 + 64,), 0xEE, dtype=torch.uint8, device="cuda")
    y = raw[:T * H * 2].view(torch.int16).view(T, H)
    q.qlin_experts_w4(dev(xb), dev(ids), dev(wt), *packed, y, work[:size])
    assert (host(raw)[-64:] == 0xEE).all() and (host(work)[-64:] == 0xEE).all(), "written past a buffer"
    return R.bf16_values(host(y))


def check(y, xb, ids, wt, ws, group):
    ref, bound = R.experts(R.bf16_values(xb), ids, wt, *ws, group)
    assert (np.abs(y - ref) <= bound + R.BF16_HALF * (np.abs(ref) + bound)).all()


CASES = [  # T, E, k, H, I, group, zeros
    (1, 1, 1, 32, 32, 32, False),
    (1, 8, 2, 128, 256, 128, True),
    (1, 64, 8, 512, 384, 128, False),
    (1, 40, 32, 96, 160, 32, True),
    (3, 16, 5, 320, 64, 64, True),
    (8, 12, 4, 256, 96, 32, False),
    (9, 12, 4, 256, 96, 32, False),
    (37, 40, 6, 352, 224, 32, True),
    (70, 3, 2, 128, 128, 128, False),
    (130, 2, 1, 192, 320, 64, True),
    (200, 7, 7, 128, 128, 64, False),
    (257, 300, 3, 64, 64, 64, True),
    (300, 4, 2, 640, 384, 128, False),
    (90, 1024, 8, 32, 32, 32, False),
]


@pytest.mark.parametrize("T,E,k,H,I,group,zeros", CASES)
def test_against_64_bits(T, E, k, H, I, group, zeros):
    case = make(1, T, E, k, H, I, group, zeros)
    print(f"experts T={T} E={E} k={k} H={H} I={I} group={group} zeros={zeros}", flush=True)
    check(run(*case), *case, group)


@pytest.mark.parametrize("T", [1, 5, 50, 400])
def test_slots_without_an_expert(T):
    """-1, E and beyond add nothing; a token without any expert gets zeros; the others are as they were."""
    E, k, H, I, group = 6, 3, 128, 128, 64
    xb, ids, wt, ws = make(2, T, E, k, H, I, group, True)
    rng = np.random.default_rng(3)
    ids = np.where(rng.random(ids.shape) < 0.3, rng.choice(np.array([-1, E, E + 100, -2 ** 31, 2 ** 31 - 1], np.int64), ids.shape),
                   ids).astype(np.int32)
    ids[T // 2] = -1
    y = run(xb, ids, wt, ws)
    check(y, xb, ids, wt, ws, group)
    assert (y[T // 2] == 0).all()


def test_nobody_wants_an_expert():
    xb, ids, wt, ws = make(4, 64, 5, 2, 64, 64, 32, False)
    assert (run(xb, np.full_like(ids, -1), wt, ws) == 0).all()


@pytest.mark.parametrize("T", [2, 100, 700])
def test_everybody_wants_one_expert(T):
    xb, ids, wt, ws = make(5, T, 9, 2, 96, 160, 32, True)
    ids[:, 0], ids[:, 1] = 7, 7            # and twice
    check(run(xb, ids, wt, ws), xb, ids, wt, ws, 32)


def test_same_bits_again_and_on_another_stream():
    torch = torch_mod()
    q = Q()
    T, k = 150, 4
    xb, ids, wt, ws = make(6, T, 16, k, 256, 192, 64, False, skew=2.0)
    packed = [q.qlin_pack_w4(dev(w[0]), dev(w[1])) for w in ws]
    x, i, w = dev(xb), dev(ids), dev(wt)
    outs = []
    streams = [None, None, torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for s in streams:                      # at the same time, each with its own workspace
        y = torch.empty((T, 256), dtype=torch.int16, device="cuda")
        work = torch.empty(q.qlin_experts_w4_workspace(T, k, *packed), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        q.qlin_experts_w4(x, i, w, *packed, y, work, stream=s)
        outs.append((y, work))
    torch.cuda.synchronize()
    for y, _ in outs[1:]:
        assert np.array_equal(host(y), host(outs[0][0]))


@pytest.mark.parametrize("T", [1, 60, 300])
def test_a_token_does_not_depend_on_its_neighbours(T):
    """NaN in one token's input reaches that token's output alone."""
    xb, ids, wt, ws = make(7, T, 4, 2, 128, 128, 128, False)
    a = run(xb, ids, wt, ws)
    bad = T // 3
    xb[bad, 5] = 0x7FC0
    b = run(xb, ids, wt, ws)
    assert np.isnan(b[bad]).all()
    keep = np.arange(T) != bad
    assert np.array_equal(a[keep], b[keep])


def layer(torch, q, xb, T, E, k, H, I, group):
    """A mixture-of-experts layer as a program runs it: router product, routing, experts' MLP, a shared dense MLP
    beside it and an output projection, all on 4-bit weights."""
    rng = np.random.default_rng(8)
    ws = {n: R.weights(rng, s, K, group, False) for n, s, K in (("router", (E,), H), ("gate", (E, I), H), ("up", (E, I), H),
                                                               ("down", (E, H), I), ("sg", (I,), H), ("su", (I,), H), ("o", (H,), I))}
    p = {n: q.qlin_pack_w4(dev(w[0]), dev(w[1])) for n, w in ws.items()}
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    t = {"x": dev(xb), "bias": dev(bias), "logits": torch.empty((T, E), device="cuda"),
         "ids": torch.empty((T, k), dtype=torch.int32, device="cuda"), "wt": torch.empty((T, k), device="cuda"),
         "y": torch.empty((T, H), dtype=torch.int16, device="cuda"), "h": torch.empty((T, I), dtype=torch.int16, device="cuda"),
         "o": torch.empty((T, H), device="cuda"),
         "work": torch.empty(q.qlin_experts_w4_workspace(T, k, p["gate"], p["up"], p["down"]), dtype=torch.uint8, device="cuda")}

    def step():
        q.qlin_linear_w4(t["x"], [(p["router"], t["logits"])], out=q.OUT_F32)
        q.qlin_route(t["logits"], t["ids"], t["wt"], score=q.SCORE_SIGMOID, bias=t["bias"], groups=4, top_groups=2, scale=2.5)
        q.qlin_experts_w4(t["x"], t["ids"], t["wt"], p["gate"], p["up"], p["down"], t["y"], t["work"])
        q.qlin_linear_swiglu_w4(t["x"], p["sg"], p["su"], t["h"])
        q.qlin_linear_w4(t["h"], [(p["o"], t["o"])], out=q.OUT_F32)
    return ws, bias, t, step


@pytest.mark.parametrize("T", [1, 48, 260])
def test_a_layer_of_them_together_eager_and_replayed(T):
    torch = torch_mod()
    q = Q()
    E, k, H, I, group = 16, 4, 256, 128, 64
    rng = np.random.default_rng(9)
    xb = R.bf16_bits(rng.standard_normal((T, H)))
    ws, bias, t, step = layer(torch, q, xb, T, E, k, H, I, group)
    step()
    torch.cuda.synchronize()
    x = R.bf16_values(xb)
    logits, ids = host(t["logits"]).copy(), host(t["ids"]).copy()
    ref, bound = R.linear(x, ws["router"], group)
    assert (np.abs(logits - ref) <= bound).all()
    rid, rw = R.route(logits, k, 1, bias, 4, 2, 2, True, 2.5)
    assert np.array_equal(ids, rid) and (np.abs(host(t["wt"]) - rw) <= 2.0 ** -23 * rw).all()
    check(R.bf16_values(host(t["y"])), xb, ids, host(t["wt"]), [ws[n] for n in ("gate", "up", "down")], group)
    hv = R.bf16_values(host(t["h"]))
    ref, bound = R.swiglu(x, ws["sg"], ws["su"], group)
    assert (np.abs(hv - ref) <= bound + R.BF16_HALF * (np.abs(ref) + bound)).all()
    ref, bound = R.linear(hv, ws["o"], group)
    assert (np.abs(host(t["o"]) - ref) <= bound).all()

    outs = [t[n] for n in ("logits", "ids", "wt", "y", "h", "o")]
    eager = [host(o).copy() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        for o in (*outs, t["work"]):
            o.view(torch.uint8).fill_(0xA5 + rep)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert np.array_equal(host(o), e), f"replay {rep} differs from the eager result"
        step()                             # eager work between the replays
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert np.array_equal(host(o), e)


@pytest.mark.parametrize("T,E,k,H,I,group,zeros", [(1, 16, 4, 256, 512, 128, False), (4, 6, 3, 128, 160, 32, True),
                                                   (30, 24, 4, 256, 320, 64, True), (90, 12, 2, 128, 256, 128, False)])
def test_few_rows_keep_16_bits_of_h(T, E, k, H, I, group, zeros):
    """Where the weights are streamed (few rows of each expert), h goes on as a bf16 value and the bf16 rounding of
    what that left: an error of at most 2^-8 * 2^-8 of h."""
    xb, ids, wt, ws = make(10, T, E, k, H, I, group, zeros)
    y = run(xb, ids, wt, ws)
    ref, bound = R.experts(R.bf16_values(xb), ids, wt, *ws, group, h_half=2.0 ** -16)
    assert (np.abs(y - ref) <= bound + R.BF16_HALF * (np.abs(ref) + bound)).all()


@pytest.mark.parametrize("T,E,k,group", [(128, 256, 4, 32), (128, 257, 4, 32), (129, 256, 4, 32), (512, 100, 1, 64), (64, 65, 8, 128),
                                         (33, 64, 15, 64), (256, 3, 2, 32)])
def test_around_the_sizes_that_need_no_sorting_launch(T, E, k, group):
    """Up to 512 slots of up to 256 experts are not sorted by a launch of their own: both sides, with ids that are no
    expert's, a skewed choice, and an expert chosen by every token."""
    H, I = 128, 256
    xb, ids, wt, ws = make(11, T, E, k, H, I, group, False, skew=3.0)
    rng = np.random.default_rng([12, T, E])
    ids = np.where(rng.random(ids.shape) < 0.1, rng.choice(np.array([-1, E, -2 ** 31, 2 ** 31 - 1], np.int64), ids.shape),
                   ids).astype(np.int32)
    ids[:, 0] = E - 1
    check(run(xb, ids, wt, ws), xb, ids, wt, ws, group)
    again = [run(xb, ids, wt, ws) for _ in range(2)]
    assert np.array_equal(again[0], again[1])
