"""A library of another ABI version is named as such, whatever symbols it lacks."""
import os
import re
import shutil
import subprocess

import pytest

Q = pytest.importorskip("quantized_linear_layers_token_amd")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_library_of_before_is_refused_by_its_version(tmp_path, monkeypatch):
    if shutil.which("gcc") is None:
        pytest.skip("gcc is not installed")
    src, out = tmp_path / "old.c", tmp_path / "libqlin.so"
    src.write_text("int qlin_abi_version(void) { return 3; }\n")      # without the symbols that came after it
    subprocess.run(["gcc", "-shared", "-fPIC", str(src), "-o", str(out)], check=True)
    monkeypatch.setattr(Q, "LIB_PATH", str(out))
    with pytest.raises(ImportError, match="ABI 3"):
        Q._load()


def test_the_4bit_calls_have_a_version_of_their_own():
    """Version 3 is the library without them."""
    text = open(os.path.join(ROOT, "include", "qlin.h")).read()
    assert int(re.search(r"#define QLIN_ABI_VERSION (\d+)", text).group(1)) > 3
