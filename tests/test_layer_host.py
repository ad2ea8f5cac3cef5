"""The norm, rotary, cache and attention entry points without a GPU: the header, the exported symbols and the binding
agree; the C-ABI layer under host sanitizers; the attention's index arithmetic in host code; the binding's own checks; the
rotary frequencies; and the matrix-core result hazard in the kernels' assembly."""
import copy
import math
import os
import pickle
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest

import test_host_sanitizers as sanitizers
import test_mfma_hazards as hazards

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = os.path.join(ROOT, "tests", "hostcheck")
CSRC = os.path.join(ROOT, "quantized_linear_layers_token_amd", "csrc")
Q = pytest.importorskip("quantized_linear_layers_token_amd")
torch = pytest.importorskip("torch")


def test_header_symbols_and_constants():
    text = open(os.path.join(ROOT, "include", "qlin_layer.h")).read()
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(qlin_[a-z0-9_]+)\s*\(", code))
    assert names == set(Q.SIGNATURES_LAYER)
    for n in names:
        assert hasattr(Q.lib(), n), f"{n} not exported by libqlin.so"
    for name, value in (("HEADS", Q.MAX_HEADS), ("HEAD_DIM", Q.MAX_HEAD_DIM)):
        assert int(re.search(rf"#define QLIN_MAX_{name} (\d+)", text).group(1)) == value
    enums = {k: int(v) for k, v in re.findall(r"(QLIN_CACHE_[A-Z0-9]+) = (\d+)", text)}
    assert enums == {"QLIN_CACHE_BF16": Q.CACHE_BF16, "QLIN_CACHE_INT8": Q.CACHE_INT8, "QLIN_CACHE_FP8": Q.CACHE_FP8}


def test_header_is_c_and_structs_match(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("gcc is not installed")
    src = tmp_path / "t.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "qlin_layer.h"\n'
                   'int main(void) { printf("%zu %zu %zu %zu %zu %zu", sizeof(qlin_rotation), sizeof(qlin_kv_cache), sizeof(qlin_queries),\n'
                   '  offsetof(qlin_rotation, strength), offsetof(qlin_kv_cache, kind), offsetof(qlin_queries, heads)); return 0; }\n')
    exe = str(tmp_path / "t")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), str(src), "-o", exe], capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stderr
    import ctypes
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    assert got == [ctypes.sizeof(Q.QlinRotation), ctypes.sizeof(Q.QlinKVCache), ctypes.sizeof(Q.QlinQueries), Q.QlinRotation.strength.offset,
                   Q.QlinKVCache.kind.offset, Q.QlinQueries.heads.offset]
    assert len(Q._PACK_QUERIES(1, 2, 3, 4, 5, 6)) == ctypes.sizeof(Q.QlinQueries)


def test_validation_layer_under_sanitizers(tmp_path):
    asan = sanitizers._asan_runtime()
    if asan is None:
        pytest.skip("g++ with AddressSanitizer is not installed")
    out = str(tmp_path / "libqlin_layer_hostcheck.so")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
           "-fPIC", "-shared", "-x", "c++", os.path.join(CSRC, "layer_api.hip"),
           "-x", "c++", os.path.join(HC, "stub_layer_launchers.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env["LD_PRELOAD"] = asan + ((" " + env["LD_PRELOAD"]) if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    r = subprocess.run([sys.executable, os.path.join(HC, "layer_validation_driver.py"), out], capture_output=True, text=True, env=env,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "no sanitizer report" in r.stdout


def test_attention_indices_in_host_code(tmp_path):
    """Bad pages, windows, ragged and empty sequences: every row that would be loaded lies in the cache, every live token
    is taken once, and there is a workgroup for every item and room for every partial sum."""
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path / "attn_index_check")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", os.path.join(HC, "attn_index_check.cpp"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and "every bound held" in r.stdout, r.stdout + r.stderr


def test_scales_are_correctly_rounded(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    exe = str(tmp_path / "rounding_check")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-mfma", "-ffp-contract=off", os.path.join(HC, "rounding_check.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip() == "0 differ", r.stdout


def t(*shape, dtype=torch.int16):
    return torch.zeros(shape, dtype=dtype)


def rejects(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


def test_binding_checks():
    """Wrong tensors raise ValueError before the library sees an address (host tensors: nothing could be launched)."""
    i8, u8, i32, f32, f16 = torch.int8, torch.uint8, torch.int32, torch.float32, torch.float16
    # norm
    x, g, q, s = t(3, 128), t(128), t(3, 128, dtype=i8), t(3, dtype=f32)
    rejects("x must be", Q.qlin_norm_int8, t(3, 128, dtype=f32), g, q, s)
    rejects("x must be", Q.qlin_norm_int8, t(128, 3).t(), g, q, s)
    rejects("gamma must be", Q.qlin_norm_int8, x, t(64), q, s)
    rejects("not float16", Q.qlin_norm_int8, x, t(128, dtype=f16), q, s)
    rejects("q must be", Q.qlin_norm_int8, x, g, t(2, 128, dtype=i8), s)
    rejects("s must be", Q.qlin_norm_int8, x, g, q, t(4, dtype=f32))
    rejects("s must be", Q.qlin_norm_fp8, x, g, q, s, group=128)
    rejects("come together", Q.qlin_norm_int8, x, g, q, s, residual=x)
    rejects("come together", Q.qlin_norm_bf16, x, g, t(3, 128), sum_out=x)
    rejects("residual must be", Q.qlin_norm_bf16, x, g, t(3, 128), residual=t(3, 64), sum_out=x)
    rejects("sum_out must be", Q.qlin_norm_bf16, x, g, t(3, 128), residual=x, sum_out=t(6, 64))
    rejects("device tensors", Q.qlin_norm_int8, x, g, q, s, stream=0)
    rejects("device tensors", Q.qlin_norm_bf16, x, g, t(3, 128), stream=0)
    # rope
    rope = Q.Rope(32, device="cpu")
    h, pos = t(5, 4, 64), t(5, dtype=i32)
    rejects("x must be", Q.qlin_rope, t(5, 64), pos, rope, h)
    rejects("x must be", Q.qlin_rope, t(5, 4, 64, dtype=f32), pos, rope, h)
    rejects("not float16", Q.qlin_rope, t(5, 4, 64, dtype=f16), pos, rope, h)
    rejects("contiguous", Q.qlin_rope, t(5, 64, 4).transpose(1, 2), pos, rope, h)
    rejects("y must be", Q.qlin_rope, h, pos, rope, t(5, 3, 64))
    rejects("positions must be", Q.qlin_rope, h, pos.long(), rope, h)
    rejects("positions must be", Q.qlin_rope, h, t(4, dtype=i32), rope, h)
    rejects("gamma must be", Q.qlin_rope, h, pos, rope, h, gamma=t(32))
    rejects("device tensors", Q.qlin_rope, h, pos, rope, h, stream=0)
    # cache
    k = t(7, 2, 16, 64, dtype=i8)
    ks = t(7, 2, 16, dtype=f32)
    rejects("k and v must be", Q.KVCache, t(7, 2, 64, dtype=i8), t(7, 2, 64, dtype=i8), ks, ks)
    rejects("k and v must be", Q.KVCache, k, k.view(u8), ks, ks)
    rejects("k and v must be", Q.KVCache, k.float(), k.float(), ks, ks)
    rejects("v must be", Q.KVCache, k, t(7, 2, 16, 32, dtype=i8), ks, ks)
    rejects("k_scale must be", Q.KVCache, k, k)
    rejects("v_scale must be", Q.KVCache, k, k, ks, ks[:6])
    rejects("v_scale must be", Q.KVCache, k, k, ks, ks.int())
    rejects("no scales", Q.KVCache, k.bfloat16(), k.bfloat16(), ks, ks)
    rejects("dtype must be", Q.KVCache.empty, 1, 1, 16, 64, torch.float16, "cpu")
    cache = Q.KVCache(k, k.clone(), ks, ks.clone())
    with pytest.raises(AttributeError, match="cannot be replaced"):
        cache.k = k
    slots, kv = t(5, dtype=i32), t(5, 2, 64)
    rejects("slots must be", Q.qlin_cache_write, cache, slots.long(), kv, kv)
    rejects("slots must be", Q.qlin_cache_write, cache, t(5, 1, dtype=i32), kv, kv)
    rejects("k must be", Q.qlin_cache_write, cache, slots, t(5, 3, 64), kv)
    rejects("v must be", Q.qlin_cache_write, cache, slots, kv, t(4, 2, 64))
    rejects("come together", Q.qlin_cache_write, cache, slots, kv, kv, rope=rope)
    rejects("positions must be", Q.qlin_cache_write, cache, slots, kv, kv, rope=rope, positions=t(4, dtype=i32))
    rejects("k_gamma must be", Q.qlin_cache_write, cache, slots, kv, kv, k_gamma=t(32))
    rejects("with q_out", Q.qlin_cache_write, cache, slots, kv, kv, rope=rope, positions=pos, q=h)
    rejects("rope or q_gamma", Q.qlin_cache_write, cache, slots, kv, kv, q=h, q_out=h)
    rejects("q_out must be", Q.qlin_cache_write, cache, slots, kv, kv, rope=rope, positions=pos, q=h, q_out=t(5, 3, 64))
    rejects("need q", Q.qlin_cache_write, cache, slots, kv, kv, q_gamma=t(64))
    rejects("device tensors", Q.qlin_cache_write, cache, slots, kv, kv, rope=rope, positions=pos, q=h, q_out=h, stream=0)
    rejects("k must be", Q.qlin_cache_read, cache, slots, t(4, 2, 64), kv)
    rejects("v must be", Q.qlin_cache_read, cache, slots, kv, kv.float())
    rejects("device tensors", Q.qlin_cache_read, cache, slots, kv, kv.clone(), stream=0)
    # attention
    need = Q.qlin_attn_decode_workspace(8, cache)
    assert need > 0
    with pytest.raises(Q.QlinError):
        Q.qlin_attn_decode_workspace(7, cache)
    q, out, pages, lengths, work = t(3, 8, 64), t(3, 8, 64), t(3, 4, dtype=i32), t(3, dtype=i32), t(need, dtype=u8)
    rejects("q must be", Q.qlin_attn_decode, t(3, 512), cache, pages, lengths, out, work)
    rejects("q must be", Q.qlin_attn_decode, t(3, 8, 32), cache, pages, lengths, out, work)
    rejects("out must be", Q.qlin_attn_decode, q, cache, pages, lengths, out[:2], work)
    rejects("pages must be", Q.qlin_attn_decode, q, cache, pages.long(), lengths, out, work)
    rejects("pages must be", Q.qlin_attn_decode, q, cache, pages[:2], lengths, out, work)
    rejects("lengths must be", Q.qlin_attn_decode, q, cache, pages, lengths.long(), out, work)
    rejects("workspace holds", Q.qlin_attn_decode, q, cache, pages, lengths, out, work[:-1])
    rejects("device tensors", Q.qlin_attn_decode, q, cache, pages, lengths, out, work, stream=0)


def test_descriptions_copied_and_pickled_hold_their_own_addresses():
    cache = Q.KVCache.empty(3, 2, 16, 64, torch.int8, "cpu")
    rope = Q.Rope(32, 5e5, interleaved=True, strength=1.25, device="cpu")
    for again in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        c = Q.QlinKVCache.from_buffer_copy(again._bytes)
        assert (c.k, c.v, c.k_scale, c.v_scale) == tuple(x.data_ptr() for x in (again.k, again.v, again.k_scale, again.v_scale))
        assert again.k.data_ptr() != cache.k.data_ptr() and (c.pages, c.kv_heads, c.page_size, c.dim, c.kind) == (3, 2, 16, 64, Q.CACHE_INT8)
    for again in (copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
        c = Q.QlinRotation.from_buffer_copy(again._bytes)
        assert c.frequencies == again.frequencies.data_ptr() != rope.frequencies.data_ptr()
        assert (c.dims, c.interleaved, c.strength) == (32, 1, 1.25) and torch.equal(again.frequencies, rope.frequencies)
    for kind, code in ((torch.bfloat16, Q.CACHE_BF16), (torch.uint8, Q.CACHE_FP8), (torch.float8_e4m3fn, Q.CACHE_FP8)):
        assert Q.KVCache.empty(1, 1, 16, 16, kind, "cpu").kind == code


def test_rotary_frequencies():
    plain = Q.Rope(128, 5e5, device="cpu").frequencies.numpy()
    assert plain.shape == (64,) and plain.dtype == np.float64
    assert np.allclose(plain, 5e5 ** (-np.arange(64) / 64), rtol=1e-14)
    assert np.allclose(Q.Rope(128, 5e5, "linear", 4.0, device="cpu").frequencies.numpy(), plain / 4, rtol=1e-14)
    ntk = Q.Rope(64, 1e4, "ntk", 8.0, device="cpu").frequencies.numpy()
    # the fastest pair stays, the slowest is stretched by the factor: that is what the base is chosen for
    assert abs(ntk[0] - 1) < 1e-14 and abs(ntk[-1] / (1e4 ** (-62 / 64) / 8) - 1) < 1e-12
    bands = Q.Rope(128, 5e5, "bands", 8.0, 8192, device="cpu")
    turns = 8192 * plain / (2 * math.pi)
    for f, p, n in zip(bands.frequencies.numpy(), plain, turns):
        if n >= 4:
            assert abs(f / p - 1) < 1e-14
        elif n <= 1:
            assert abs(f * 8 / p - 1) < 1e-14
        else:
            w = (n - 1) / 3
            assert abs(f - (p * w + p / 8 * (1 - w))) < 1e-14 * p
    assert bands.strength == 1.0 and (turns > 4).any() and (turns < 1).any()
    yarn = Q.Rope(128, 1e6, "yarn", 4.0, 32768, device="cpu")
    p = 1e6 ** (-np.arange(64) / 64)
    ratio = yarn.frequencies.numpy() / p
    turns = 32768 * p / (2 * math.pi)
    assert np.allclose(ratio[turns > 40], 1) and np.allclose(ratio[turns < 0.8], 0.25) and (np.diff(ratio) <= 1e-12).all()
    assert abs(yarn.strength - (0.1 * math.log(4) + 1)) < 1e-15
    given = torch.linspace(1, 2, 16, dtype=torch.float64)
    assert torch.equal(Q.Rope(32, frequencies=given).frequencies, given)
    rejects("multiple of 16", Q.Rope, 24, device="cpu")
    rejects("multiple of 16", Q.Rope, 272, device="cpu")
    rejects("base must be", Q.Rope, 32, base=0.5, device="cpu")
    rejects("base must be", Q.Rope, 32, factor=math.inf, device="cpu")
    rejects("scaling must be", Q.Rope, 32, scaling="other", device="cpu")
    rejects("needs the original", Q.Rope, 32, scaling="yarn", factor=2.0, device="cpu")
    rejects("needs the original", Q.Rope, 32, scaling="bands", factor=2.0, original=4096, fast=1.0, device="cpu")
    rejects("frequencies must be", Q.Rope, 32, frequencies=given.float())
    rejects("frequencies must be", Q.Rope, 64, frequencies=given)


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_every_mfma_result_access_is_padded(tmp_path):
    b = hazards._load_build()
    flags = [f for f in b.CFLAGS if f != "-fPIC"]
    text = hazards._asm("attn_decode.hip", str(tmp_path), flags, b.hipcc())
    assert sum(1 for op, _ in hazards._parse(text)[0] if op.startswith("v_mfma")) > 100
    bad = hazards.violations(text)
    assert not bad, bad[:5]
    spills = [int(v) for v in re.findall(r"\.vgpr_spill_count:\s+(\d+)", text)]
    assert max(spills) == 0
    assert not re.search(r"v_pk_(add|mul|fma)_f32", text)
    lost = lost_registers(text)
    assert not lost, lost[:5]


def lost_registers(text):
    """Byte permutations between a kernel's first and last matrix instruction that read a register which f32 arithmetic
    wrote last: there they transpose loaded values, and the register allocator has been seen to give the upper half of a
    loaded pair away before its use."""
    arithmetic = ("v_sub_f32", "v_add_f32", "v_mul_f32", "v_exp_f32", "v_lshlrev_b32", "v_cvt_pk_bf16_f32", "v_fma_f32")
    found = []
    for name, body in re.findall(r"^(_ZN4qlin\S*attn_kernel\S*):(.*?)s_endpgm", text, re.M | re.S):
        code = [line.strip() for line in body.splitlines() if line.startswith("\t") and not line.strip().startswith((".", ";"))]
        products = [i for i, line in enumerate(code) if line.startswith("v_mfma")]
        if not products:
            continue
        wrote = {}
        for line in code[products[0]:products[-1]]:
            op = line.split()[0]
            args = [a.strip() for a in line[len(op):].split(",")]
            if op == "v_perm_b32":
                found += [(name, line) for a in args[1:3] if wrote.get(a, "").startswith(arithmetic)]
            pair = re.match(r"v\[(\d+):(\d+)\]$", args[0])
            for r in (range(int(pair[1]), int(pair[2]) + 1) if pair else ()):
                wrote[f"v{r}"] = op
            if re.match(r"v\d+$", args[0]):
                wrote[args[0]] = op
    return found


def test_the_scan_for_lost_registers_finds_one():
    kernel = "_ZN4qlin1_attn_kernel:\n\tv_mfma_f32 v[0:3], v[4:7], v[8:11], v[0:3]\n\tglobal_load_dwordx2 v[20:21], v[2:3], off\n"
    used = "\tv_perm_b32 v30, v20, v21, s1\n\tv_mfma_f32 v[0:3], v[4:7], v[8:11], v[0:3]\n\ts_endpgm\n"
    assert not lost_registers(kernel + used)
    assert lost_registers(kernel + "\tv_sub_f32_e32 v21, v1, v2\n" + used)
