"""The choice of the heads' kernel on the host: every form that the library holds is taken by some call, and by those of the
GPU tests against the definition."""
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
    return lib


def built(source, kernel, tmp_path):
    """Template arguments of every form of a kernel, from the assembly of the source as the library is built from it."""
    b = hazards._load_build()
    if not os.path.exists(b.hipcc()):
        pytest.skip("hipcc is not installed")
    text = hazards._asm(source, str(tmp_path), [f for f in b.CFLAGS if f != "-fPIC"], b.hipcc())
    forms = re.findall(rf"^_ZN4qlin12_GLOBAL__N_1{len(kernel)}{kernel}I((?:L[ib]\d+E)+)E\S*:", text, re.M)
    assert forms
    return {tuple(int(v) for v in re.findall(r"L[ib](\d+)E", f)) for f in forms}


def heads_form(rules, kind, T, heads, kv_heads, dim, dims, interleaved):
    lanes = rules.heads_lanes(dim)
    return lanes, KINDS.index(kind), int(dims > 0), int(dims > 0 and interleaved), rules.heads_tokens(lanes, heads + 2 * kv_heads, T)


def test_every_form_of_the_heads_kernel_is_taken(rules, tmp_path):
    taken = set()
    for T, dim, kv_heads, heads in itertools.product((1, 1023, 1024, 8191, 8192, 1 << 24), range(16, 257, 16), (0, 1, 2, 8), (0, 1, 2, 3, 8, 32)):
        for turn in (0, 1, 2):      # none, halves, neighbours
            if kv_heads:
                taken |= {heads_form(rules, kind, T, heads, kv_heads, dim, 16 * (turn > 0), turn == 2) for kind in KINDS}
            elif heads and turn:
                taken.add(heads_form(rules, "bf16", T, heads, 0, dim, 16, turn == 2))
    assert taken == built("heads.hip", "heads_kernel", tmp_path)


def test_the_gpu_tests_take_every_form_of_the_heads_kernel(rules, tmp_path):
    taken = {heads_form(rules, "bf16", T, heads, 0, dim, dims, interleaved) for T, heads, dim, dims, interleaved, _ in F.ROPE}
    taken |= {heads_form(rules, kind, T, heads, kv_heads, dim, dims, interleaved)
              for T, heads, kv_heads, dim, _, dims, interleaved, _ in F.WRITE for kind in KINDS}
    assert taken == built("heads.hip", "heads_kernel", tmp_path)
