"""Host-only checks of the operators around the linears: symbols, frequencies of the
rotation, what is refused (before any HIP call), workspace sizes, and the reference's own
gradient against differences."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import decoder_abi as dec
import decoder_ref as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qlora_decoder.h")
SOME = ctypes.c_void_p(4096)          # aligned, never followed: every call below is refused on the host
ARG, UNSUPPORTED, WORKSPACE = nf4.NF4_ERR_ARG, nf4.NF4_ERR_UNSUPPORTED, nf4.NF4_ERR_WORKSPACE


def test_declared_symbols_are_exported():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(qlora_\w+)\s*\(", text)))
    assert names == ["qlora_head_loss", "qlora_head_loss_workspace_bytes", "qlora_kv_append", "qlora_kv_attention",
                     "qlora_kv_attention_workspace_bytes", "qlora_rope_apply"]
    for n in names:
        assert hasattr(nf4.load_library(), n)


@pytest.mark.parametrize("rotary", [2, 64, 128, 22])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=2.0),
                                dict(scaling="parts", factor=8.0, original_length=4096), dict(base=500000.0)])
def test_frequencies(rotary, kw):
    if kw.get("scaling") == "ntk" and rotary == 2:
        pytest.skip("ntk scaling needs four values")
    plan = nf4.rope_plan(rotary, device="cpu", **kw)
    theta, magnitude = ref.theta_of(rotary, **kw)
    turns = plan.freq.numpy().astype(np.float64) / 2.0 ** 64
    # a frequency is a float64 quotient cut to 2^-64 of a turn
    assert np.all(np.abs(turns - theta / (2 * math.pi)) <= 2.0 ** -52)
    assert plan.magnitude == pytest.approx(magnitude, abs=1e-15)


def test_frequency_refusals():
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, scaling="cubic"), dict(rotary_dim=8, factor=0.0),
                dict(rotary_dim=8, scaling="parts", factor=2.0), dict(rotary_dim=2, scaling="ntk", factor=2.0),
                dict(rotary_dim=8, base=float("inf"))):
        with pytest.raises(ValueError):
            nf4.rope_plan(device="cpu", **bad)


def heads(n=4, dim=128, data=4096, token_stride=None, head_stride=None):
    return dec._Heads(data, n * dim if token_stride is None else token_stride, dim if head_stride is None else head_stride, n)


def rope_status(rope=None, M=4, dim=128, dtype=nf4.NF4_BF16, ins=None, outs=None, count=1, positions=SOME):
    rope = rope or dec._Rope(4096, 128, 0, 1.0)
    ins, outs = ins or heads(), outs or heads(data=8192)
    return dec._library().qlora_rope_apply(ctypes.byref(rope), 0, positions, M, dim, dtype, ctypes.byref(ins),
                                           ctypes.byref(outs), count, None)


def test_rope_refusals():
    assert rope_status(M=0) == nf4.NF4_OK
    assert rope_status(M=-1) == UNSUPPORTED and rope_status(M=1 << 24) == UNSUPPORTED
    assert rope_status(dim=1024) == UNSUPPORTED
    assert rope_status(dtype=7) == ARG and rope_status(count=3) == ARG and rope_status(positions=None) == ARG
    for bad in (dec._Rope(None, 128, 0, 1.0), dec._Rope(4096, 127, 0, 1.0), dec._Rope(4096, 130, 0, 1.0),
                dec._Rope(4096, 0, 0, 1.0), dec._Rope(4096, 128, 0, float("nan"))):
        assert rope_status(rope=bad) == ARG
    assert rope_status(ins=heads(data=None)) == ARG and rope_status(ins=heads(data=4097)) == ARG
    assert rope_status(outs=heads(n=5, data=8192)) == ARG and rope_status(ins=heads(head_stride=64)) == ARG
    assert rope_status(outs=heads(data=4096, token_stride=1024)) == ARG      # in place with other strides
    assert "strides" in nf4.load_library().nf4_last_error().decode()


def test_rope_refuses_rows_that_share_memory():
    for out in (heads(data=8192, token_stride=0), heads(data=8192, token_stride=64), heads(data=8192, token_stride=511),
                heads(data=8192, token_stride=128, head_stride=511), heads(data=8192, token_stride=0, head_stride=512),
                heads(n=1, data=8192, token_stride=127)):
        n = out.heads
        assert rope_status(ins=heads(n), outs=out) == ARG
        assert "overlap" in nf4.load_library().nf4_last_error().decode()
        out.data = 4096
        assert rope_status(ins=out, outs=out) == ARG                              # in place
    both = (dec._Heads * 2)(heads(), heads())
    assert dec._library().qlora_rope_apply(ctypes.byref(dec._Rope(4096, 128, 0, 1.0)), 0, SOME, 4, 128, nf4.NF4_BF16, both, both, 2, None) == ARG
    assert "same" in nf4.load_library().nf4_last_error().decode()


def cache(**kw):
    a = dict(codes=4096, scales=4096, pages=10, kv_heads=4, page_size=16, head_dim=128)
    a.update(kw)
    return dec._Cache(*a.values())


def batch(**kw):
    a = dict(starts=4096, lengths=4096, table=4096, table_stride=4, tokens=3, seqs=2, table_width=4)
    a.update(kw)
    return dec._Batch(*a.values())


def append_status(c=None, b=None, k=None, v=None, rope=None, q=None, qo=None):
    by = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return dec._library().qlora_kv_append(by(c or cache()), by(b or batch()), by(k or heads()), by(v or heads()), by(rope),
                                          by(q), by(qo), None)


def test_append_refusals():
    assert append_status(b=batch(tokens=0)) == nf4.NF4_OK
    for c, want in ((cache(head_dim=96), UNSUPPORTED), (cache(page_size=24), UNSUPPORTED), (cache(page_size=512), UNSUPPORTED),
                    (cache(codes=None), ARG), (cache(codes=4100), ARG), (cache(scales=None), ARG), (cache(kv_heads=0), ARG),
                    (cache(pages=0), UNSUPPORTED), (cache(pages=1 << 30), UNSUPPORTED)):
        assert append_status(c=c) == want
    for b, want in ((batch(tokens=-1), UNSUPPORTED), (batch(tokens=1 << 23), UNSUPPORTED), (batch(seqs=0), ARG),
                    (batch(seqs=70000), UNSUPPORTED), (batch(starts=None), ARG), (batch(lengths=None), ARG),
                    (batch(table=None), ARG), (batch(table_stride=3), ARG), (batch(starts=4097), ARG),
                    (batch(table_width=1 << 28, table_stride=1 << 28), UNSUPPORTED)):
        assert append_status(b=b) == want
    assert append_status(k=heads(n=3)) == ARG and append_status(v=heads(n=5)) == ARG
    assert append_status(k=heads(token_stride=513)) == ARG and append_status(v=heads(data=4104)) == ARG
    assert append_status(q=heads(n=8)) == ARG and append_status(q=heads(n=8), qo=heads(n=4, data=8192)) == ARG
    assert append_status(rope=dec._Rope(4096, 256, 0, 1.0)) == ARG


def test_append_and_attention_refuse_rows_that_share_memory():
    for out in (heads(n=8, data=8192, token_stride=0), heads(n=8, data=8192, token_stride=512), heads(n=8, data=8192, token_stride=128, head_stride=128)):
        assert append_status(q=heads(n=8), qo=out) == ARG and "overlap" in nf4.load_library().nf4_last_error().decode()
        assert attention_status(out=out, length=100000) == ARG and "overlap" in nf4.load_library().nf4_last_error().decode()
    assert attention_status(out=heads(n=8, data=8192, token_stride=128, head_stride=384), length=100000) == WORKSPACE


def attention_status(c=None, b=None, q=None, out=None, scale=0.1, new=1, length=64, ws=None, wsb=0):
    by = ctypes.byref
    return dec._library().qlora_kv_attention(by(c or cache()), by(b or batch()), by(q or heads(n=8)), by(out or heads(n=8, data=8192)),
                                             scale, new, length, ws, wsb, None)


def test_attention_refusals():
    assert attention_status(b=batch(tokens=0)) == nf4.NF4_OK
    assert attention_status(q=heads(n=6)) == ARG and attention_status(out=heads(n=4)) == ARG
    assert attention_status(scale=float("nan")) == ARG and attention_status(new=0) == ARG and attention_status(length=0) == ARG
    assert attention_status(new=1 << 23) == UNSUPPORTED and attention_status(length=1 << 31) == UNSUPPORTED
    size = dec._library().qlora_kv_attention_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch()), 8, 1, 100000)
    assert size > 0
    assert attention_status(length=100000) == WORKSPACE
    assert attention_status(length=100000, ws=SOME, wsb=size - 1) == WORKSPACE
    assert attention_status(length=100000, ws=ctypes.c_void_p(4096 + 16), wsb=size) == ARG


def test_attention_workspace_holds_the_parts_and_no_more():
    # 24 single tokens of 64 heads of 128 behind up to 4096 keys: a sum of 128 values and two statistics for each of up to
    # four chunks of a row
    size = dec._library().qlora_kv_attention_workspace_bytes(
        ctypes.byref(cache(kv_heads=64, page_size=64)), ctypes.byref(batch(tokens=24, seqs=24, table_stride=64, table_width=64)), 64, 1, 4096)
    assert 0 < size <= 24 * 64 * 4 * (128 + 2) * 4 + 256


def test_attention_plans_for_the_batch_it_has():
    size = lambda tokens, new: dec._library().qlora_kv_attention_workspace_bytes(  # noqa: E731
        ctypes.byref(cache()), ctypes.byref(batch(tokens=tokens)), 8, new, 100000)
    for tokens in (1, 3, 100, 1000):
        assert size(tokens, tokens) == size(tokens, 1000 * tokens) == size(tokens, (1 << 23) - 1) > 0
    assert attention_status(c=cache(kv_heads=1024, pages=8), b=batch(seqs=40000), q=heads(n=1024), out=heads(n=1024, data=8192)) == UNSUPPORTED
    assert "2^25" in nf4.load_library().nf4_last_error().decode()


def test_attention_scale_refusals():
    for scale in (float("inf"), -float("inf"), 2.0 ** 127, -3e38):
        assert attention_status(scale=scale) == ARG
        assert "scale" in nf4.load_library().nf4_last_error().decode()
    assert attention_status(scale=-1.7e38, length=100000) == WORKSPACE       # below 2^127: the next check is met


def loss_status(X=SOME, M=8, K=64, W=SOME, V=100, t=SOME, dl=SOME, loss=SOME, dX=SOME, dW=SOME, ws=SOME, wsb=1 << 40):
    return dec._library().qlora_head_loss(X, M, K, W, V, t, -100, dl, loss, dX, dW, ws, wsb, None)


def test_loss_refusals():
    assert loss_status(M=0, dW=None) == nf4.NF4_OK
    assert loss_status(M=-1) == ARG and loss_status(V=0) == ARG and loss_status(K=0) == ARG
    assert loss_status(K=72) == UNSUPPORTED and loss_status(K=1 << 20) == UNSUPPORTED
    assert loss_status(M=1 << 22) == UNSUPPORTED and loss_status(V=1 << 23) == UNSUPPORTED
    assert loss_status(X=None) == ARG and loss_status(W=None) == ARG and loss_status(t=None) == ARG
    assert loss_status(dl=None) == ARG and loss_status(loss=None, dX=None, dW=None) == ARG
    odd = ctypes.c_void_p(4100)
    assert loss_status(X=odd) == ARG and loss_status(dX=odd) == ARG and loss_status(dW=odd) == ARG and loss_status(t=odd) == ARG
    need = dec._library().qlora_head_loss_workspace_bytes(8, 64, 100, 1, 1)
    assert need > 0 and loss_status(wsb=need - 1) == WORKSPACE and loss_status(ws=None) == WORKSPACE
    assert loss_status(ws=ctypes.c_void_p(4096 + 64)) == ARG


def test_loss_workspace_does_not_hold_the_logits():
    M, V, K = 4096, 128000, 4096
    assert dec._library().qlora_head_loss_workspace_bytes(M, K, V, 1, 0) < M * V * 2 / 4


@pytest.mark.parametrize("dx,dw", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("M", [1, 33, 64, 100, 512, 2048, 4096, 5000, 131072, 200000])
def test_loss_workspace_is_what_the_header_says(M, dx, dw):
    up = lambda n, to: -(-n // to) * to  # noqa: E731
    for K in (64, 512, 4096, 8192):
        for V in (1, 500, 32000, 128256, 131200):
            m = up(M, 512)
            v = min(max(512, (1 << 27) // (2 * m) // 512 * 512), up(V, 512))
            pieces = -(-V // v)
            kept = dw and 2 * m * v * pieces <= 1 << 30
            least = 2 * m * K + (2 * m * v if dx or dw else 0) + 2 * M * K * dw + (3 * m * v * pieces if kept else 0)
            rows = 64 * m + 4 * m * (pieces + 1)                                # statistics of rows
            most = least + 8 * m * up(-(-min(V, v if dx or dw else V) // 32), 4) + 4 * M * K * 64 * dx + rows + 16 * 256
            size = dec._library().qlora_head_loss_workspace_bytes(M, K, V, dx, dw)
            assert least <= size <= most, (M, K, V, dx, dw, least, size, most)


def test_tensor_refusals_without_a_gpu():
    plan = nf4.rope_plan(8, device="cpu")
    x = torch.zeros((2, 1, 8))
    for call in (lambda: nf4.rope_fwd(plan, torch.zeros(2, dtype=torch.int32), x),
                 lambda: nf4.head_loss(x[0].bfloat16(), x[0].bfloat16(), torch.zeros(1, dtype=torch.int64))):
        with pytest.raises(ValueError):
            call()


def test_reference_gradient_against_differences():
    g = torch.Generator().manual_seed(3)
    X, W = torch.randn((3, 5), generator=g).double(), torch.randn((7, 5), generator=g).double()
    t, dl = torch.tensor([2, -100, 6]), torch.tensor([0.5, 1.0, -2.0]).double()
    _, dX, dW, _, _ = ref.head_loss(X, W, t, dl)
    f = lambda x, w: (ref.head_loss(x, w, t, dl)[0] * dl).sum()  # noqa: E731
    for A, d, of in ((X, dX, lambda a: f(a, W)), (W, dW, lambda a: f(X, a))):
        for i in range(A.shape[0]):
            for j in range(A.shape[1]):
                e = torch.zeros_like(A)
                e[i, j] = 1e-6
                # central differences: error of about 1e-12 f''' + 1e-16 / 1e-6
                assert abs((of(A + e) - of(A - e)) / 2e-6 - d[i, j]) < 1e-8


@pytest.mark.parametrize("M,V,K", [(384, 3000, 64), (33, 4000, 128)])
def test_the_limit_on_dw_tells_kept_bits_from_lost_ones(M, V, K):
    # dW as the library makes it: exponentials kept in 24 bits, G and dW rounded to bf16
    g = torch.Generator().manual_seed(M)
    X = torch.randn((M, K), generator=g).bfloat16()
    W = (torch.randn((V, K), generator=g) / math.sqrt(K)).bfloat16()
    t, dl = torch.randint(0, V // 2, (M,), generator=g), torch.randn(M, generator=g) / M
    _, _, dW, _, z = ref.head_loss(X, W, t, dl)
    z = z / math.log(2)
    R, lse = torch.round(z[torch.arange(M), t]), torch.logsumexp(z * math.log(2), 1) / math.log(2)
    E = torch.exp2(z - R[:, None]).float()
    factor = (dl / dl.abs().max()).double() * torch.exp2(R - lse)
    error = {}
    for low in ("right", "zero", "misplaced"):
        G = (ref.kept_exponentials(E, low).double() * factor[:, None]).bfloat16().double()
        got = (G.t() @ X.double() * dl.abs().max().double()).bfloat16().double()
        error[low] = float((got - dW)[V // 2:].norm() / dW[V // 2:].norm())
    assert error["right"] <= ref.DW_NORM < error["zero"] and ref.DW_NORM < error["misplaced"], error


def test_reference_rotation_against_differences():
    # the gradient of sum(w . rotate(x)) by differences is rotate-back of w
    theta, mag = ref.theta_of(6, scaling="parts", factor=4.0, original_length=64)
    r = np.random.RandomState(0)
    x, w = r.randn(2, 1, 8), r.randn(2, 1, 8)
    back = ref.rotate(w, [5, 900], 6, True, theta, mag, back=True)
    f = lambda a: (w * ref.rotate(a, [5, 900], 6, True, theta, mag)).sum()  # noqa: E731
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-5
        assert abs((f(x + e) - f(x - e)) / 2e-5 - back[i]) < 1e-9


def test_reference_codes():
    v = ref.e4m3_values()
    assert v[126] == 448 and v[1] == 2.0 ** -9 and np.isnan(v[127])
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.nan_to_num(t, nan=1e9), np.nan_to_num(v, nan=1e9))
    x = np.concatenate([v[:127], (v[:126] + v[1:127]) / 2, np.linspace(-448, 448, 4001)])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_nearest(x.astype(np.float32)), want)
