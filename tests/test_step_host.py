"""Host-only checks of the operators of include/qlora_step.h: symbols, what is refused (before any HIP call), workspace
sizes, and the reference's own gradients against differences."""
import ctypes
import os
import re

import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import step_abi as abi
import step_ref as ref
from decoder_abi import _Batch, _Cache, _Heads

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qlora_step.h")
SOME, MORE, THIRD, FOURTH = 4096, 8192, 12288, 16384       # aligned, never followed: every call below is refused on the host
OK, ARG, UNSUPPORTED, WORKSPACE = nf4.NF4_OK, nf4.NF4_ERR_ARG, nf4.NF4_ERR_UNSUPPORTED, nf4.NF4_ERR_WORKSPACE
F32, BF16 = nf4.NF4_F32, nf4.NF4_BF16


def by(x):
    return None if x is None else ctypes.byref(x)


def why():
    return nf4.load_library().nf4_last_error().decode()


def test_declared_symbols_are_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qlora_\w+)\s*\(", text)))
    assert names == ["qlora_adamw_step_paged_scaled", "qlora_adamw_step_scaled", "qlora_block_norm_bwd",
                     "qlora_block_norm_bwd_workspace_bytes", "qlora_block_norm_fwd", "qlora_grad_clip",
                     "qlora_grad_clip_workspace_bytes", "qlora_grad_norm", "qlora_grad_norm_workspace_bytes",
                     "qlora_kv_attention_window", "qlora_kv_attention_window_workspace_bytes", "qlora_logits_shape"]
    for n in names:
        assert hasattr(nf4.load_library(), n)


def norm(**kw):
    a = dict(pre=None, post=None, gate=None, gate_rows=1, norm_pre=1, norm_post=0, dtype=BF16, scale=1.0, eps=1e-6)
    a.update(kw)
    return abi.Norm(*a.values())


def rows(data=SOME, stride=64):
    return abi.Rows(data, stride)


def fwd(n=None, M=4, K=64, dtype=BF16, h=rows(), x=rows(MORE), h_out=rows(THIRD), y=rows(FOURTH)):
    return abi.library().qlora_block_norm_fwd(by(n or norm()), M, K, dtype, by(h), by(x), by(h_out), by(y), None)


def bwd(n=None, M=4, K=64, dtype=BF16, h=rows(), x=rows(MORE), dy=rows(20480), dh=None, dh_out=rows(THIRD), dx=rows(FOURTH), dpre=None,
        dpost=None, dgate=None, ws=None, size=0):
    return abi.library().qlora_block_norm_bwd(by(n or norm()), M, K, dtype, by(h), by(x), by(dy), by(dh), by(dh_out), by(dx), dpre, dpost,
                                              dgate, ws, size, None)


def test_block_norm_refusals():
    assert fwd(M=0) == OK
    assert fwd(M=-1) == UNSUPPORTED and fwd(M=1 << 31) == UNSUPPORTED and fwd(K=0) == UNSUPPORTED and fwd(K=32769) == UNSUPPORTED
    assert abi.library().qlora_block_norm_fwd(None, 4, 64, BF16, by(rows()), None, None, by(rows(MORE)), None) == ARG
    for n in (norm(eps=0.0), norm(eps=1e-39), norm(eps=float("inf")), norm(scale=float("nan")), norm(dtype=5), norm(pre=SOME, norm_pre=0), norm(post=SOME),
              norm(pre=4097), norm(gate=SOME, gate_rows=0), norm(gate=SOME, gate_rows=3), norm(gate=SOME, gate_rows=8)):
        assert fwd(n) == ARG and bwd(n) == ARG, why()
    assert fwd(dtype=9) == ARG and bwd(dtype=9) == ARG
    for bad in (None, rows(None), rows(4097), rows(stride=63), rows(stride=-64)):
        assert fwd(h=bad) == ARG and bwd(h=bad) == ARG
    for bad in (None, rows(None), rows(stride=0)):
        assert fwd(h_out=bad) == ARG and fwd(y=bad) == ARG and bwd(dh_out=bad) == ARG and bwd(dx=bad) == ARG
    # without a block: nothing that belongs to one
    assert fwd(x=None) == ARG and fwd(norm(norm_post=1), x=None, h_out=None) == ARG and fwd(norm(gate=SOME), x=None, h_out=None) == ARG
    assert fwd(norm(norm_pre=0), x=None, h_out=None, y=None) == ARG
    assert fwd(norm(norm_pre=0)) == ARG and bwd(norm(norm_pre=0)) == ARG                     # y (dy) where there is no norm
    # memory that is written
    assert fwd(h_out=rows(SOME, 128)) == ARG and "stride" in why()
    assert fwd(h_out=rows(MORE)) == ARG and fwd(y=rows(SOME)) == ARG and fwd(y=rows(THIRD)) == ARG and fwd(y=rows(MORE)) == ARG
    assert bwd(dh=rows(THIRD, 128)) == ARG and bwd(dh_out=rows(MORE)) == ARG and bwd(dx=rows(20480)) == ARG and bwd(dx=rows(THIRD)) == ARG
    assert bwd(dh=rows(FOURTH)) == ARG
    # gradients of weights that are not there, and the workspace
    assert bwd(dpre=SOME) == ARG and bwd(dpost=SOME) == ARG and bwd(dgate=SOME) == ARG and bwd(norm(pre=SOME), dpre=4098) == ARG
    need = abi.library().qlora_block_norm_bwd_workspace_bytes(4000, 64, 1, 1, 0, 0)
    assert need > 0
    assert bwd(norm(pre=SOME), M=4000, dpre=MORE) == WORKSPACE
    assert bwd(norm(pre=SOME), M=4000, dpre=MORE, ws=SOME, size=need - 1) == WORKSPACE
    assert bwd(norm(pre=SOME), M=4000, dpre=MORE, ws=4100, size=need) == ARG


def test_block_norm_workspace():
    bytes_of = abi.library().qlora_block_norm_bwd_workspace_bytes
    for M in (1, 5, 100, 4097, 1 << 20):
        for K in (1, 64, 1000, 8192, 32768):
            assert bytes_of(M, K, 1, 0, 0, 0) == 0 and bytes_of(M, K, M, 0, 0, 1) == 0
            one = bytes_of(M, K, 1, 1, 0, 0)
            assert one % 256 == 0 and one <= 2048 * K * 4 + 256 and bytes_of(M, K, 1, 1, 1, 1) <= 4 * one + 256
            assert one <= bytes_of(M, K, 1, 1, 1, 0) <= bytes_of(M, K, 1, 1, 1, 1)
    assert bytes_of(-1, 64, 1, 1, 1, 1) == bytes_of(4, 0, 1, 1, 1, 1) == bytes_of(4, 40000, 1, 1, 1, 1) == 0


def tensors(*t):
    return (abi.Tensor * len(t))(*[abi.Tensor(*x) for x in t])


def test_gradient_refusals():
    L = abi.library()
    good = tensors((SOME, 100, F32), (MORE, 100, BF16), (None, 0, F32))
    size = L.qlora_grad_norm_workspace_bytes(good, 3)
    assert size > 0 and size % 256 == 0
    norm_of = lambda g=good, n=3, m=1.0, out=SOME, f=MORE, ws=SOME, b=size: L.qlora_grad_norm(g, n, m, out, f, ws, b, None)  # noqa: E731
    assert norm_of(n=-1) == UNSUPPORTED and norm_of(n=(1 << 24) + 1) == UNSUPPORTED and norm_of(g=None) == ARG
    assert norm_of(out=None) == ARG and norm_of(out=4097) == ARG and norm_of(f=4098) == ARG
    assert norm_of(m=-0.5) == ARG and norm_of(m=float("nan")) == ARG
    assert norm_of(ws=None) == WORKSPACE and norm_of(b=size - 1) == WORKSPACE and norm_of(ws=4100) == ARG
    for bad in ((None, 5, F32), (4098, 5, F32), (4097, 5, BF16), (SOME, -1, F32), (SOME, 5, 3), (SOME, (1 << 40) + 1, F32)):
        assert norm_of(tensors(bad), 1) == ARG and L.qlora_grad_norm_workspace_bytes(tensors(bad), 1) == 0
    scale = lambda g, o, m=1.0, out=SOME, ws=SOME, b=1 << 20: L.qlora_grad_clip(g, o, len(o), m, out, ws, b, None)  # noqa: E731
    a, b = (4 << 20, 100, F32), (8 << 20, 50, BF16)
    assert scale(tensors(a), tensors((8 << 20, 99, F32))) == ARG and scale(tensors(a), tensors((8 << 20, 100, BF16))) == ARG
    assert scale(tensors(a), tensors(a), out=None) == ARG and scale(tensors(a), tensors(a), out=4097) == ARG
    assert scale(tensors(a), tensors(a), m=-1.0) == ARG and scale(tensors(a), tensors(a), m=float("nan")) == ARG
    size = L.qlora_grad_clip_workspace_bytes(tensors(a), 1)
    assert scale(tensors(a), tensors(a), ws=None) == WORKSPACE and scale(tensors(a), tensors(a), b=size - 1) == WORKSPACE
    assert scale(tensors(a), tensors(a), ws=4100) == ARG
    inside = ((4 << 20) + 4, 10, F32)
    far = (12 << 20, 10, F32)
    for g, o in (((a, a), (a, a)), ((a, inside), (a, inside)), ((a, far), (a, inside)), ((a, inside), (a, far)), ((a,), (((4 << 20) - 4, 100, F32),)),
                 ((b, a, far), (b, far, far))):
        assert scale(tensors(*g), tensors(*o)) == ARG, (g, o)


def test_logit_refusals():
    def call(rows_=3, V=100, dtype=F32, z=abi.Rows(SOME, 100), out=abi.Rows(MORE, 100), **kw):
        r = dict(history=None, history_stride=8, history_width=8, lengths=None, prompts=None, repetition=1.0, presence=0.0, frequency=0.0,
                 repetitions=None, presences=None, frequencies=None, bias_ids=None, bias_ids_stride=4, bias=None, bias_stride=4, biases=4,
                 allowed=None, allowed_stride=4)
        r.update(kw)
        return abi.library().qlora_logits_shape(by(abi.Rules(*r.values())), rows_, V, dtype, by(z), by(out), None)
    assert call(rows_=0) == OK
    assert abi.library().qlora_logits_shape(None, 3, 100, F32, by(rows()), by(rows(MORE)), None) == ARG
    assert call(rows_=-1) == UNSUPPORTED and call(rows_=1 << 24) == UNSUPPORTED and call(V=0) == UNSUPPORTED and call(V=1 << 28) == UNSUPPORTED
    for bad in (dict(dtype=4), dict(z=None), dict(z=abi.Rows(SOME, 99)), dict(z=abi.Rows(4098, 100)), dict(out=abi.Rows(MORE, 0)),
                dict(out=abi.Rows(SOME, 101)), dict(history=SOME, history_stride=7), dict(history=SOME, history_width=-1),
                dict(history=SOME, history_width=(1 << 31) - 1, history_stride=1 << 40), dict(history=4097), dict(lengths=SOME), dict(prompts=SOME),
                dict(history=SOME, repetition=0.0), dict(history=SOME, repetition=float("nan")), dict(history=SOME, presence=float("inf")),
                dict(history=SOME, frequency=float("nan")), dict(bias_ids=SOME), dict(bias=SOME), dict(bias_ids=SOME, bias=SOME, bias_stride=3),
                dict(bias_ids=SOME, bias=SOME, bias_ids_stride=3), dict(bias_ids=SOME, bias=SOME, biases=-1), dict(allowed=SOME, allowed_stride=3),
                dict(allowed=4098), dict(history=SOME, repetitions=4097)):
        assert call(**bad) == ARG, (bad, why())


def test_window_refusals():
    c, b = _Cache(SOME, SOME, 10, 4, 16, 128), _Batch(SOME, SOME, SOME, 4, 3, 2, 4)
    q, out = (_Heads(at, 8 * 128, 128, 8) for at in (SOME, MORE))
    call = lambda w, s, ws=None: abi.library().qlora_kv_attention_window(by(c), by(b), by(q), by(out), 0.1, 2, 64, w, s, ws, 0, None)  # noqa: E731
    size = lambda w, s, longest=64, batch=b: abi.library().qlora_kv_attention_window_workspace_bytes(by(c), by(batch), 8, 1, longest, w, s)  # noqa: E731
    for w, s in ((0, 0), (-1, 0), (1 << 31, 0), (1, -1), (1, (1 << 30) + 1)):
        assert call(w, s) == ARG and size(w, s) == 0
    # the window, not the sequence, sizes the chunks: a long sequence's workspace stops growing
    many = _Batch(SOME, SOME, SOME, 1 << 20, 3, 3, 1 << 20)
    plain = abi.library().qlora_kv_attention_workspace_bytes(by(c), by(many), 8, 1, 1 << 24)
    assert size(4096, 4, 1 << 24, many) == size(4096, 4, 1 << 20, many) < plain


@pytest.mark.parametrize("pre,post,gate,later", [(True, None, None, True), ("w", "w", 3, True), ("w", True, "one", False), (None, "w", 6, True), ("w", None, 1, False)])
def test_reference_gradients_against_differences(pre, post, gate, later):
    # a change of d in one number moves L = sum(dy y) + sum(dh h') by d times its gradient, within d^2 of the curvature: 1e-6
    g = torch.Generator().manual_seed(5)
    rand = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    M, K = 6, 9
    t = dict(h=rand(M, K), x=rand(M, K))
    w = lambda v: 1 + 0.3 * rand(K) if v == "w" else v  # noqa: E731
    how = dict(pre=w(pre), post=w(post), gate=None if gate is None else rand(K) if gate == "one" else rand(gate, K))
    dy, dh = (rand(M, K) if pre is not None else None), (rand(M, K) if later else None)

    def loss(h, x, **kw):
        s, y = ref.block_norm(h, x, scale=0.7, eps=1e-2, **kw)
        return float((0 if dy is None else (dy * y(s)).sum()) + (0 if dh is None else (dh * s).sum()))

    new, _ = ref.block_norm(t["h"], t["x"], scale=0.7, eps=1e-2, **how)
    got, _ = ref.block_norm_back(new, dy, dh, t["x"], scale=0.7, eps=1e-2, **how)
    named = {"dh": "h", "dx": "x", "dpre": "pre", "dpost": "post", "dgate": "gate"}
    for name, of in named.items():
        v = {**t, **how}[of]
        assert (name in got) == torch.is_tensor(v)
        if name not in got:
            continue
        for _ in range(12):
            at = tuple(int(torch.randint(0, n, (1,), generator=g)) for n in v.shape)
            values = []
            for d in (1e-4, -1e-4):
                u = v.clone()
                u[at] += d
                values.append(loss(**{**t, **how, of: u}))
            assert abs((values[0] - values[1]) / 2e-4 - float(got[name][at])) <= 1e-6
