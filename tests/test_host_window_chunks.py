"""The chunks of attention with a window stay short enough for a batch with a single long sequence: compiled against the header
that the library's launcher uses."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_nf4_quantized_09_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_window_chunks(tmp_path):
    exe = tmp_path / "window_chunks_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-I", CSRC, os.path.join(HERE, "c", "window_chunks_check.cpp"), "-o", str(exe)], check=True)
    sizes, bad = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert sizes > 10000 and bad == 0
