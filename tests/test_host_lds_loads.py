"""Wait states around the direct loads into LDS, in the assembly that hipcc makes of the kernels.

On gfx950 a load into LDS reads M0, which needs a wait state after a scalar write of M0, and a memory
instruction needs five between a vector instruction's write of a scalar register and its reading it.
hipcc looks after both for its own instructions, not for strings of assembly: this reads what it made
of head_loss.hip, whose loads into LDS are such strings.  A branch target between the write and the
load is passed as if the code ran straight through it."""
import os
import re
import shutil
import subprocess

import pytest

from bit_nf4_quantized_09_amd import build

FROM_SCALAR, FROM_VECTOR = 1, 5


def registers(text):
    """The scalar registers named in an operand list."""
    found = {int(n) for n in re.findall(r"\bs(\d+)\b", text)}
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        found |= set(range(int(a), int(b) + 1))
    return found


def instructions(text):
    lines = (line.split(";")[0].strip() for line in text.splitlines())
    return [x for x in lines if x and not x.startswith(".") and not x.endswith(":")]


def wait_states(x):
    m = re.match(r"s_nop (\d+)", x)
    return int(m.group(1)) + 1 if m else 1


def short_waits(code):
    """(loads into LDS, those with too few wait states before them)."""
    loads, short = 0, []
    for i, x in enumerate(code):
        if not (re.match(r"(buffer|global)_load", x) and re.search(r"\blds\b", x)):
            continue
        loads += 1
        reads, passed = registers(x), 0
        for y in reversed(code[max(0, i - FROM_VECTOR):i]):
            if y.startswith("s_mov_b32 m0") and passed < FROM_SCALAR:
                short.append((y, x))
            if y.startswith("v_") and passed < FROM_VECTOR and registers(y.split(",")[0]) & reads:
                short.append((y, x))
            passed += wait_states(y)
    return loads, short


def test_the_reader_finds_what_it_looks_for():
    load = "buffer_load_dwordx4 v1, s[4:7], s9 offen lds"
    assert short_waits(["s_mov_b32 m0, s3", load])[1]
    assert not short_waits(["s_mov_b32 m0, s3", "s_nop 0", load])[1]
    assert short_waits(["v_readfirstlane_b32 s9, v2", "s_mov_b32 m0, s3", "s_nop 2", load])[1]
    assert not short_waits(["v_readfirstlane_b32 s9, v2", "s_mov_b32 m0, s3", "s_nop 3", load])[1]
    assert not short_waits(["v_readfirstlane_b32 s8, v2", "s_nop 0", load])[1]
    assert short_waits(["v_readfirstlane_b32 s6, v2", "s_nop 1", load])[1]


@pytest.mark.skipif(shutil.which(build.HIPCC) is None, reason="needs hipcc")
def test_loads_into_lds_have_their_wait_states(tmp_path):
    out = tmp_path / "head_loss.s"
    subprocess.run([build.HIPCC] + build.FLAGS + ["-S", "--cuda-device-only", os.path.join(build.CSRC, "head_loss.hip"),
                                                  "-o", str(out)], check=True, capture_output=True)
    loads, short = short_waits(instructions(out.read_text()))
    assert loads > 100
    assert not short, (len(short), short[:3])
