"""The experts' call captured once and replayed on other inputs, another routing among them: one token after the other,
rows found by the workgroups, sorted by a launch, and tiled.  Equality with the exact results."""
import numpy as np
import pytest

import w4_exact as X
import w4_reference as R
from gpu_helpers import dev, host, torch_mod
from test_w4_linear_gpu import Q, pack

pytestmark = pytest.mark.gpu

CASES = [X.LOW[2], X.LOW[3], X.LOW[6], X.MANY[1], X.MANY[8], X.MANY[9]]


@pytest.mark.parametrize("case", CASES)
def test_replayed_on_other_inputs(case):
    torch = torch_mod()
    T, E, k, H, I = case[:5]
    x, ids, wt, ws = X.experts_case(2, *case, False)
    packed = [pack(w) for w in ws]
    t = {"x": dev(R.bf16_bits(x).reshape(T, H)), "ids": dev(ids), "wt": dev(wt)}
    y = torch.empty((T, H), dtype=torch.int16, device="cuda")
    work = torch.empty(Q().qlin_experts_w4_workspace(T, k, *packed), dtype=torch.uint8, device="cuda")

    def step():
        Q().qlin_experts_w4(t["x"], t["ids"], t["wt"], *packed, y, work)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    rng = np.random.default_rng(40)
    for rep in range(4):
        rows = rng.permutation(T)
        if rep == 1:                                  # every token to one expert
            new_ids = np.where(np.arange(k) == 0, E - 1, -1)[None].repeat(T, 0).astype(np.int32)
        elif rep == 2:                                # nobody to any
            new_ids = np.full((T, k), -1, np.int32)
        else:
            new_ids = np.where(rng.random((T, k)) < 0.2, E + 5, rng.permuted(ids, axis=1)[rows]).astype(np.int32)
        new_x = x[rows]
        for name, value in (("x", R.bf16_bits(new_x).reshape(T, H)), ("ids", new_ids)):
            t[name].copy_(dev(value))
        want = X.experts(new_x, np.where(new_ids < E, new_ids, -1), wt, ws, 2) if (new_ids < E).any() else np.zeros((T, H))
        want = R.bf16_values(R.bf16_bits(want)).reshape(T, H)
        print(f"replay {rep} of {case}", flush=True)
        for run in (graph.replay, step):              # and an eager call between the replays, in the same workspace
            y.fill_(-1)
            work.fill_(0xEE)
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            assert np.array_equal(R.bf16_values(host(y)), want), (rep, run)
