"""The check that lets parts of one packed tensor through, compiled for the host (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_operands_that_interleave_are_apart(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "overlap_check"
    src = os.path.join(ROOT, "tests", "native", "overlap_check.cpp")
    inc = os.path.join(ROOT, "tiled_attention_08_gb300", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", inc, src, "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout
