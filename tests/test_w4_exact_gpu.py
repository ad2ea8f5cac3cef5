"""SwiGLU and the experts' MLP on 4-bit weights where every result is exact: equality, in every form, whatever the order
of the sums.  The low part of h: results made of nothing else.  And many rows of each expert on random inputs."""
import numpy as np
import pytest

import w4_exact as X
import w4_reference as R
from gpu_helpers import dev, host
from test_experts_gpu import check, make, run
from test_w4_linear_gpu import Q, check_guard, outputs, pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,I,K,group,zeros", X.SWIGLU)
def test_swiglu(M, I, K, group, zeros):
    x, gate, up = X.swiglu_case(1, M, I, K, group, zeros)
    (h,), raw = outputs(M, [I], False)
    print(f"exact swiglu M={M} I={I} K={K} group={group} zeros={zeros}", flush=True)
    Q().qlin_linear_swiglu_w4(dev(R.bf16_bits(x)), pack(gate), pack(up), h)
    assert np.array_equal(host(h).view(np.uint16), R.bf16_bits(X.swiglu(x, gate, up)[0]).reshape(M, I))
    check_guard(raw)


def experts_equal(case, low):
    print(f"exact experts {case} low={low}", flush=True)
    x, ids, wt, ws = X.experts_case(2, *case, low)
    y = run(R.bf16_bits(x), ids, wt, ws)
    assert np.array_equal(y, R.bf16_values(R.bf16_bits(X.experts(x, ids, wt, ws, 2))).reshape(y.shape))


@pytest.mark.parametrize("case", X.ANY)
def test_experts(case):
    experts_equal(case, False)


@pytest.mark.parametrize("case", X.LOW)
def test_few_rows_keep_both_parts_of_h(case):
    experts_equal(case, True)


@pytest.mark.parametrize("case", X.MANY)
def test_many_rows_against_64_bits(case):
    T, E, k, H, I, group, zeros = case
    print(f"experts {case}", flush=True)
    inputs = make(3, T, E, k, H, I, group, zeros, skew=1.0)
    check(run(*inputs), *inputs, group)
