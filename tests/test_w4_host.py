"""The 4-bit, routing and experts entry points without a GPU: the header, the exported symbols and the binding agree;
the C-ABI layer under host sanitizers; the binding's own checks; and the matrix-core result hazard in the new kernels'
assembly."""
import hashlib
import json
import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest

import test_host_sanitizers as sanitizers
import test_mfma_hazards as hazards

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HC = os.path.join(ROOT, "tests", "hostcheck")
Q = pytest.importorskip("quantized_linear_layers_token_amd")


def test_header_symbols_and_constants():
    text = open(os.path.join(ROOT, "include", "qlin_w4.h")).read()
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(qlin_[a-z0-9_]+)\s*\(", code))
    assert names == set(Q.SIGNATURES_W4)
    for n in names:
        assert hasattr(Q.lib(), n), f"{n} not exported by libqlin.so"
    for name, value in (("EXPERTS", Q.MAX_EXPERTS), ("CHOICES", Q.MAX_CHOICES), ("GROUPS", Q.MAX_GROUPS)):
        assert int(re.search(rf"#define QLIN_MAX_{name} (\d+)", text).group(1)) == value
    enums = {k: int(v) for k, v in re.findall(r"(QLIN_SCORE_[A-Z]+) = (\d+)", text)}
    assert enums == {"QLIN_SCORE_SOFTMAX": Q.SCORE_SOFTMAX, "QLIN_SCORE_SIGMOID": Q.SCORE_SIGMOID}


def test_header_is_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "qlin_w4.h"\nint main(void) { qlin_w4_weight w = {0}; return (int)w.n; }\n')
    if shutil.which("gcc") is None:
        pytest.skip("gcc is not installed")
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I" + os.path.join(ROOT, "include"), "-c", str(src), "-o",
                        str(tmp_path / "t.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_validation_layer_under_sanitizers(tmp_path):
    asan = sanitizers._asan_runtime()
    if asan is None:
        pytest.skip("g++ with AddressSanitizer is not installed")
    out = str(tmp_path / "libqlin_w4_hostcheck.so")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + os.path.join(ROOT, "include"),
           "-fPIC", "-shared", "-x", "c++", os.path.join(ROOT, "quantized_linear_layers_token_amd", "csrc", "w4_api.hip"),
           "-x", "c++", os.path.join(HC, "stub_w4_launchers.cpp"), "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ)
    env["LD_PRELOAD"] = asan + ((" " + env["LD_PRELOAD"]) if env.get("LD_PRELOAD") else "")
    env["ASAN_OPTIONS"] = "detect_leaks=0:halt_on_error=1"
    env["UBSAN_OPTIONS"] = "halt_on_error=1:print_stacktrace=1"
    r = subprocess.run([sys.executable, os.path.join(HC, "w4_validation_driver.py"), out], capture_output=True, text=True,
                       env=env, timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    assert "no sanitizer report" in r.stdout


def test_binding_checks():
    """Wrong tensors raise ValueError before the library sees an address (host tensors: nothing could be launched)."""
    import torch

    def t(*shape, dtype=torch.int16):
        return torch.zeros(shape, dtype=dtype)

    def weight(N=16, K=128, group=128, experts=1, device="cpu"):
        w = Q.W4Weight(t(64, dtype=torch.uint8), t(64), None, experts, N, K, group)
        return w

    def rejects(match, fn, *a, **k):
        with pytest.raises(ValueError, match=match):
            fn(*a, **k)

    u8, i32, f32 = torch.uint8, torch.int32, torch.float32
    # packing
    rejects("q_w must be", Q.qlin_pack_w4, t(64, dtype=u8), t(1))
    rejects("group must be", Q.qlin_pack_w4, t(16, 64, dtype=u8), t(16, 3))
    rejects("q_w must be a contiguous", Q.qlin_pack_w4, t(16, 64), t(16, 1))
    rejects("s_w must be a contiguous", Q.qlin_pack_w4, t(16, 64, dtype=u8), t(8, 1))
    rejects("z_w must be a contiguous", Q.qlin_pack_w4, t(16, 64, dtype=u8), t(16, 1), t(16, 2, dtype=u8))
    rejects("not float16", Q.qlin_pack_w4, t(16, 64, dtype=u8), t(16, 1, dtype=torch.float16))
    rejects("device tensors", Q.qlin_pack_w4, t(16, 64, dtype=u8), t(16, 1))
    # projections
    w = weight()
    rejects("one to 4", Q.qlin_linear_w4, t(2, 128), [])
    rejects("one to 4", Q.qlin_linear_w4, t(2, 128), [(w, t(2, 16))] * 5)
    rejects("x must be", Q.qlin_linear_w4, t(2, 128, dtype=f32), [(w, t(2, 16))])
    rejects("x must be", Q.qlin_linear_w4, t(2, 128, dtype=torch.float16), [(w, t(2, 16))])
    rejects("inputs", Q.qlin_linear_w4, t(2, 256), [(w, t(2, 16))])
    rejects("y must be", Q.qlin_linear_w4, t(2, 128), [(w, t(3, 16))])
    rejects("y must be", Q.qlin_linear_w4, t(2, 128), [(w, t(2, 16))], out=Q.OUT_F32)
    rejects("y must be", Q.qlin_linear_w4, t(2, 128), [(w, t(16, 2).t())])
    rejects("one matrix", Q.qlin_linear_w4, t(2, 128), [(weight(experts=2), t(2, 16))])
    rejects("group size", Q.qlin_linear_w4, t(2, 128), [(w, t(2, 16)), (weight(group=64), t(2, 16))])
    rejects("device tensors", Q.qlin_linear_w4, t(2, 128), [(w, t(2, 16))], stream=0)
    rejects("one matrix each", Q.qlin_linear_swiglu_w4, t(2, 128), w, weight(N=32), t(2, 16))
    rejects("h must be", Q.qlin_linear_swiglu_w4, t(2, 128), w, w, t(2, 32))
    # routing
    ids, wt = t(2, 4, dtype=i32), t(2, 4, dtype=f32)
    rejects("logits must be", Q.qlin_route, t(2, 8), ids, wt)
    rejects("logits must be", Q.qlin_route, t(8, 2, dtype=f32).t(), ids, wt)
    rejects("ids must be", Q.qlin_route, t(2, 8, dtype=f32), ids.long(), wt)
    rejects("ids must be", Q.qlin_route, t(3, 8, dtype=f32), ids, wt)
    rejects("weights must be", Q.qlin_route, t(2, 8, dtype=f32), ids, t(2, 3, dtype=f32))
    rejects("bias must be", Q.qlin_route, t(2, 8, dtype=f32), ids, wt, bias=t(8))
    rejects("bias must be", Q.qlin_route, t(2, 8, dtype=f32), ids, wt, bias=t(7, dtype=f32))
    # experts
    gate, down = weight(N=256, K=128, experts=4), weight(N=128, K=256, experts=4)
    size = Q.qlin_experts_w4_workspace(2, 4, gate, gate, down)
    assert size > 0
    y, work = t(2, 128), t(size, dtype=u8)
    rejects("up must have", Q.qlin_experts_w4, t(2, 128), ids, wt, gate, weight(N=128, experts=4), down, y, work)
    rejects("up must have", Q.qlin_experts_w4, t(2, 128), ids, wt, gate, gate, gate, y, work)
    rejects("ids must be", Q.qlin_experts_w4, t(2, 128), ids.long(), wt, gate, gate, down, y, work)
    rejects("y must be", Q.qlin_experts_w4, t(2, 128), ids, wt, gate, gate, down, t(2, 256), work)
    rejects("workspace holds", Q.qlin_experts_w4, t(2, 128), ids, wt, gate, gate, down, y, work[:-1])
    rejects("device tensors", Q.qlin_experts_w4, t(2, 128), ids, wt, gate, gate, down, y, work, stream=0)


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_every_mfma_result_access_is_padded(tmp_path):
    b = hazards._load_build()
    flags = [f for f in b.CFLAGS if f != "-fPIC"]
    sources = ["w4_stream.hip", "w4_tiled.hip"]
    with ThreadPoolExecutor(2) as ex:
        texts = list(ex.map(lambda s: hazards._asm(s, str(tmp_path), flags, b.hipcc()), sources))
    for src, text in zip(sources, texts):
        assert sum(1 for op, _ in hazards._parse(text)[0] if op.startswith("v_mfma")) > 1000
        bad = hazards.violations(text)
        assert not bad, f"{src}: {bad[:5]}"
        spills = [int(v) for v in re.findall(r"\.vgpr_spill_count:\s+(\d+)", text)]
        assert max(spills) <= 16, f"{src}: {max(spills)} registers spilled"


def test_measured_traffic_still_belongs_to_its_sources():
    """The bench reports the measured bytes of the decode launch only while the sources they belong to are unchanged:
    what the 4-bit calls need is declared apart from them."""
    with open(os.path.join(ROOT, "profiles", "linear_decode_int8_llama8b_traffic.json")) as f:
        recorded = json.load(f)["sources_sha256"]
    for name, sha in recorded.items():
        with open(os.path.join(ROOT, "quantized_linear_layers_token_amd", "csrc", name), "rb") as f:
            assert hashlib.sha256(f.read()).hexdigest() == sha, name
