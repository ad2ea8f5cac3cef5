"""Codes and scales of the norm and the cache over the mantissas of an absmax that bf16 rows and products give."""
import numpy as np
import pytest

import layer_reference as R
from gpu_helpers import dev, host, torch_mod

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_every_mantissa_of_an_absmax(kind):
    """t = r * gamma reaches every product of two 8-bit mantissas: rows (r, gamma) over all of them, and the codes of the
    other channels of the row, as IEEE steps in NumPy give them."""
    import quantized_linear_layers_token_amd as q
    torch = torch_mod()
    M, K = 128, 128 * 128
    # row m: r is 1 + m / 128 in the first channel of each group of 128, smaller values behind; group j: gamma 1 + j / 128
    rng = np.random.default_rng(1)
    r = rng.uniform(-0.9, 0.9, (M, 128, 128))
    r[:, :, 0] = (1 + np.arange(M) / 128)[:, None]
    g = np.repeat(1 + np.arange(128) / 128, 128)
    xb, gb = R.bits(r.reshape(M, K)), R.bits(g)
    for shift in (0, -40, -75, 30):
        sb = R.bits(R.value(xb) * 2.0 ** shift)
        if kind == "fp8":
            y = torch.empty((M, K), dtype=torch.uint8, device="cuda")
            s = torch.empty((M, 128), device="cuda")
            q.qlin_norm_fp8(dev(sb), dev(gb), y, s, group=128)
            import oracle as O
            got = O.e4m3_decode(host(y)).reshape(M, 128, 128)
            want, _ = R.codes((R.value(sb) * g).reshape(M, 128, 128), "fp8")
        else:   # one absmax to a row
            flat = sb.reshape(M * 128, 128)
            cache = q.KVCache.empty(M * 128 // 16, 1, 16, 128, torch.int8)
            t = R.bits(R.value(flat))
            at = dev(np.arange(M * 128, dtype=np.int32))
            q.qlin_cache_write(cache, at, dev(t.reshape(M * 128, 1, 128)), dev(t.reshape(M * 128, 1, 128)))
            got = host(cache.k).reshape(M * 128, 128).astype(np.float64)
            want, scale = R.codes(R.value(t), "int8")
            assert np.array_equal(host(cache.k_scale).reshape(-1), scale)
        assert np.array_equal(got, want), shift
