"""Operands of include/qlora_step.h that share memory with one that is written are refused on the host, before any HIP call,
also where they begin at different addresses; operands side by side in one buffer do not share any."""
import ctypes
import os
import shutil
import subprocess

import pytest

import bit_nf4_quantized_09_amd as nf4
import step_abi as abi
from test_step_host import SOME, bwd, fwd, norm, rows, why

ARG = nf4.NF4_ERR_ARG
HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "bit_nf4_quantized_09_amd", "csrc")
FAR = 1 << 24                  # (never followed, like SOME: every call below is refused)
ROW = 64 * 2                   # 4 rows of 64 values of bf16 are 512 bytes


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_against_a_mark_on_every_byte(tmp_path):
    exe = tmp_path / "overlap_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", CSRC, os.path.join(HERE, "c", "overlap_check.cpp"), "-o", str(exe)], check=True)
    pairs, bad = map(int, subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split())
    assert pairs > 100000 and bad == 0


def refused(status):
    assert status == ARG and "shares memory" in why(), why()


@pytest.mark.parametrize("shift", [-3 * ROW, -ROW, -2, 2, ROW, 3 * ROW, 3 * ROW + ROW - 2])
def test_norms_of_shifted_rows(shift):
    at = rows(SOME + shift)
    # in place: the stream's rows, and the block's output a row (or a value) on
    refused(fwd(x=at, h_out=rows()))
    refused(fwd(y=at, h_out=rows()))
    refused(fwd(h_out=at))                                    # shifted against the stream itself
    refused(fwd(y=at))
    for weights in (dict(pre=SOME + 512 + shift), dict(post=SOME + 512 + shift, norm_post=1), dict(gate=SOME + 512 + shift)):
        if -3 * ROW <= shift < 0:                             # a row of weights in the last rows of the stream
            refused(fwd(norm(**weights), h_out=rows()))
            refused(bwd(norm(**weights), dh_out=rows(), h=rows(FAR)))
    for name in ("h", "x", "dy", "dh", "dx"):
        refused(bwd(dh_out=rows(FAR), **{name: rows(FAR + shift)}))
        if name != "dx":
            refused(bwd(dx=rows(FAR), **{name: rows(FAR + shift)}))


def test_norms_with_strides():
    refused(fwd(h=rows(SOME, 200), h_out=rows(SOME, 200), x=rows(SOME + 137 * 2, 200)))       # one value into the row after
    refused(fwd(h=rows(SOME, 100), h_out=rows(SOME, 100), x=rows(SOME + 62 * 2, 100)))
    refused(fwd(h_out=rows(FAR, 64), x=rows(FAR + 3 * ROW, 0)))                                       # one row for all
    refused(fwd(h_out=rows(FAR, 64), x=rows(FAR + 64, 1000)))


def test_norms_weights_gradients_and_workspace():
    n = norm(pre=FAR, post=FAR + 4096, norm_post=1, gate=FAR + 8192)
    at = dict(dpre=2 * FAR, dpost=2 * FAR + 4096, dgate=2 * FAR + 8192, ws=3 * FAR, size=1 << 20)
    size = 4 * 64                                             # of each
    outputs = ("dpre", "dpost", "dgate")
    for a in outputs:
        for b in outputs:
            if a != b:
                refused(bwd(n, **{**at, a: at[b] + size - 4}))
        for where in (SOME, 20480, 8192, 12288, 16384, FAR, FAR + 4096, FAR + 8192):          # h, dy, x, dh_out, dx and the weights
            refused(bwd(n, **{**at, a: where + 4}))
    need = 1 << 24
    many = dict(M=4000, h=rows(1 << 27), x=rows(1 << 28), dy=rows(1 << 29), dh_out=rows(1 << 30), dx=rows(1 << 31))
    for where in (1 << 27, 1 << 28, 1 << 29, 1 << 30, 1 << 31, FAR, 2 * FAR):
        refused(bwd(n, **{**many, **at, "ws": where, "size": need}))


def test_logits_and_their_rules():
    rule = dict(history=None, history_stride=8, history_width=8, lengths=None, prompts=None, repetition=1.0, presence=0.0, frequency=0.0,
                repetitions=None, presences=None, frequencies=None, bias_ids=None, bias_ids_stride=4, bias=None, bias_stride=4, biases=4,
                allowed=None, allowed_stride=4)

    def call(z, out, **kw):
        r = abi.Rules(*{**rule, **kw}.values())
        return abi.library().qlora_logits_shape(ctypes.byref(r), 3, 100, nf4.NF4_F32, ctypes.byref(z), ctypes.byref(out), None)
    at = abi.Rows(FAR, 100)                                   # 1200 bytes
    for shift in (-1196, -400, -4, 4, 400, 1196):
        refused(call(abi.Rows(FAR + shift, 100), at))
    refused(call(abi.Rows(FAR, 250), abi.Rows(FAR + 99 * 4, 250)))
    refused(call(abi.Rows(FAR + 800, 0), at))                 # one row for all
    # the rules' tables, which begin before the logits and end in them: in place
    history = dict(history=2 * FAR)
    for name, size, kw in (("history", 3 * 32, {}), ("lengths", 12, history), ("prompts", 12, history), ("repetitions", 12, history),
                           ("presences", 12, history), ("frequencies", 12, history), ("bias_ids", 48, dict(bias=2 * FAR)),
                           ("bias", 48, dict(bias_ids=2 * FAR)), ("allowed", 48, {})):
        for where in (FAR - size + 4, FAR, FAR + 1196):
            refused(call(at, at, **{**kw, name: where}))


def test_the_factor_apart_from_what_the_step_writes():
    # every workgroup reads the factor, whenever it begins
    L = nf4.load_library()
    vp = ctypes.c_void_p
    p, g, m, v, half, stage = (i << 20 for i in range(1, 7))
    how = (64, 1e-4, 0.9, 0.999, 1e-8, 0.0, 1)
    for f in (p, p + 252, m, m + 128, v + 252, half, half + 124):
        assert L.qlora_adamw_step_scaled(vp(p), vp(g), vp(m), vp(v), vp(half), *how, vp(f), None) == ARG and "factor" in why()
    for f in (stage, stage + 4092, half + 124):
        assert L.qlora_adamw_step_paged_scaled(vp(p), vp(g), vp(m), vp(v), vp(half), *how, vp(f), vp(stage), 4096, None) == ARG and "factor" in why()
