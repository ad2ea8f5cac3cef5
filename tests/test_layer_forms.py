"""The choice of the heads' and the attention's kernel on the host: every form that the library holds is taken by some call, and
by those of the GPU tests against the definition."""
import ctypes
import itertools
import os
import re
import shutil
import subprocess

import pytest

import layer_forms as F
import test_mfma_hazards as hazards

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KINDS = F.KINDS


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not installed")
    out = str(tmp_path_factory.mktemp("forms") / "liblayer_forms.so")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", os.path.join(ROOT, "tests", "hostcheck", "layer_forms.cpp"), "-o", out],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(out)
    lib.heads_tokens.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int64]
    lib.attn_alone.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    return lib


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    """Of a source and a kernel: the template arguments of every form, from the assembly as the library is built from it."""
    b = hazards._load_build()
    try:
        hipcc = b.hipcc()
    except RuntimeError:
        pytest.skip("hipcc is not installed")
    found = {}

    def of(source, kernel):
        if source not in found:
            text = hazards._asm(source, str(tmp_path_factory.mktemp("asm")), [f for f in b.CFLAGS if f != "-fPIC"], hipcc)
            forms = re.findall(rf"^_ZN4qlin12_GLOBAL__N_1{len(kernel)}{kernel}I((?:L[ib]\d+E)+)E\S*:", text, re.M)
            assert forms
            found[source] = {tuple(int(v) for v in re.findall(r"L[ib](\d+)E", f)) for f in forms}
        return found[source]

    return of


def heads_form(rules, kind, T, heads, kv_heads, dim, dims, interleaved):
    lanes = rules.heads_lanes(dim)
    return lanes, KINDS.index(kind), int(dims > 0), int(dims > 0 and interleaved), rules.heads_tokens(lanes, heads + 2 * kv_heads, T)


def test_every_form_of_the_heads_kernel_is_taken(rules, built):
    taken = set()
    for T, dim, kv_heads, heads in itertools.product((1, 1023, 1024, 8191, 8192, 1 << 24), range(16, 257, 16), (0, 1, 2, 8), (0, 1, 2, 3, 8, 32)):
        for turn in (0, 1, 2):      # none, halves, neighbours
            if kv_heads:
                taken |= {heads_form(rules, kind, T, heads, kv_heads, dim, 16 * (turn > 0), turn == 2) for kind in KINDS}
            elif heads and turn:
                taken.add(heads_form(rules, "bf16", T, heads, 0, dim, 16, turn == 2))
    assert taken == built("heads.hip", "heads_kernel")


def test_the_gpu_tests_take_every_form_of_the_heads_kernel(rules, built):
    taken = {heads_form(rules, "bf16", T, heads, 0, dim, dims, interleaved) for T, heads, dim, dims, interleaved, _ in F.ROPE}
    taken |= {heads_form(rules, kind, T, heads, kv_heads, dim, dims, interleaved)
              for T, heads, kv_heads, dim, _, dims, interleaved, _ in F.WRITE for kind in KINDS}
    assert taken == built("heads.hip", "heads_kernel")


def attn_form(rules, kind, S, heads, kv_heads, dim, page, columns):
    """-> kind, channels in registers, wavefronts, one launch."""
    groups = kv_heads * -(-heads // kv_heads // 16)
    channels, alone = rules.attn_channels(dim), rules.attn_alone(S, columns * page, groups, dim)
    return KINDS.index(kind), channels, 8 if alone and channels == 64 else 4, alone


def test_the_gpu_tests_take_every_form_of_the_attention(rules, built):
    taken = {attn_form(rules, kind, len(lengths), *case, columns) for lengths, *case, columns, _ in F.ATTENTION for kind in KINDS}
    assert taken == built("attn_decode.hip", "attn_kernel")


def test_one_launch_by_each_of_its_rules(rules):
    """The table is short; it is of a medium length and the workgroups many; the sequences are more than are scanned."""
    for channels in (64, 128, 256):
        short = 512 if channels == 64 else 256
        cases = [(len(c[0]), c[4] * c[5], c[2] * -(-c[1] // c[2] // 16), c[3]) for c in F.ATTENTION if rules.attn_channels(c[3]) == channels]
        assert any(tokens <= short for _, tokens, _, _ in cases)
        medium = [c for c in cases if c[1] > short and rules.attn_alone(*c)]
        assert medium and all(tokens <= 2048 and S * groups >= 128 for S, tokens, groups, _ in medium)
        assert any(not rules.attn_alone(*c) for c in cases)
    assert rules.attn_alone(1025, 1 << 20, 1, 128) and not rules.attn_alone(1024, 1 << 20, 1, 128)
