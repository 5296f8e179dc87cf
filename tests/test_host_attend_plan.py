"""Attention's launches are sound for every size that the entry point lets through: compiled against
the header that the library's launcher uses."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_nf4_quantized_09_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_attention_plans(tmp_path):
    exe = tmp_path / "attend_plan_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, os.path.join(HERE, "c", "attend_plan_check.cpp"), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    sizes, bad = map(int, out.split()[-2:])
    assert sizes > 10000
    assert bad == 0, out
