"""Which kernels that split their registers by role may run, and that the choice of path asks for it (CPU only)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "causal_linear_attention_attn_gb300", "csrc")
SRC = os.path.join(ROOT, "tests", "native", "register_shares_test.cpp")


def test_rule(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "register_shares_test"
    subprocess.run([cxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, SRC, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == "ok"


def test_the_choice_of_the_prefill_depends_on_it():
    """Sizes of workspaces and launches take the answer of one function, and no launch refuses by itself."""
    with open(os.path.join(CSRC, "gated_tc.cu")) as f:
        src = f.read()
    supported = src[src.index("bool gated_tc_supported("):]
    assert "shares_fit" in supported[: supported.index("\n}\n")]
    assert "cudaErrorInvalidConfiguration" not in src
    with open(os.path.join(CSRC, "gated_api.cu")) as f:
        api = f.read()
    assert len(re.findall(r"gated_tc_supported\([^)]*\)", api)) == 3  # workspace, prefill, gradient
