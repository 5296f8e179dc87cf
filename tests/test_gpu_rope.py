"""Rotary positions on the GPU against float64.

Bounds.  cos and sin are within 4e-7 (a fraction of a turn rounded to 24 bits, 1.9e-7 in the
angle, and sincospi's own rounding), products and their sum round by 2^-24 each: 1e-6 times
magnitude (|a| + |b|) covers fp32.  bf16 adds half a unit of its last place, 2^-9 of the next
power of two, at most 2^-8 of the value."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import decoder_ref as ref

pytestmark = pytest.mark.gpu
SCALED = dict(none={}, linear=dict(scaling="linear", factor=4.0), ntk=dict(scaling="ntk", factor=4.0),
              parts=dict(scaling="parts", factor=8.0, original_length=4096))


def check(y, x, positions, rotary, inter, kw, back, dtype):
    theta, mag = ref.theta_of(rotary, **kw)
    x = x.float().cpu().numpy().astype(np.float64)
    want = ref.rotate(x, positions.cpu().numpy(), rotary, inter, theta, mag, back)
    a, b = ref.pair_index(rotary, inter)
    size = np.zeros_like(x)
    size[..., a] = size[..., b] = mag * (np.abs(x[..., a]) + np.abs(x[..., b]))
    tol = 1e-6 * size + (2.0 ** -8 * np.abs(want) if dtype == torch.bfloat16 else 0)
    got = y.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(got[..., rotary:], x[..., rotary:])
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) - tol)


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rotary,scaling", [(128, 128, "none"), (128, 64, "parts"), (64, 32, "linear"), (256, 256, "ntk"),
                                                (80, 80, "none"), (128, 22, "parts"), (40, 2, "none"), (511, 510, "linear")])
def test_values(dim, rotary, scaling, inter, dtype, back):
    g = torch.Generator(device="cuda").manual_seed(dim + rotary)
    for tokens, heads, kv in ((1, 1, 1), (37, 5, 2), (1030, 3, 3)):
        q = torch.randn((tokens, heads, dim), generator=g, device="cuda").to(dtype)
        k = torch.randn((tokens, kv, dim), generator=g, device="cuda").to(dtype)
        positions = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        plan = nf4.rope_plan(rotary, interleaved=inter, **SCALED[scaling])
        call = nf4.rope_bwd if back else nf4.rope_fwd
        yq, yk = call(plan, positions, q, k)
        check(yq, q, positions, rotary, inter, SCALED[scaling], back, dtype)
        check(yk, k, positions, rotary, inter, SCALED[scaling], back, dtype)
        assert torch.equal(call(plan, positions, q), yq)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rotary", [128, 64, 6])
def test_strides_and_in_place(inter, rotary):
    g = torch.Generator(device="cuda").manual_seed(7)
    plan = nf4.rope_plan(rotary, interleaved=inter)
    positions = torch.arange(50, 69, dtype=torch.int32, device="cuda")
    for pad in (0, 8, 3):                     # 3: rows that no 16-byte vector fits
        buf = torch.randn((19, 7 * 128 + pad), generator=g, device="cuda").bfloat16()
        q = buf[:, : 4 * 128].unflatten(1, (4, 128))
        k = buf[:, 4 * 128: 7 * 128].unflatten(1, (3, 128))
        want_q, want_k = nf4.rope_fwd(plan, positions, q.contiguous(), k.contiguous())
        yq, yk = nf4.rope_fwd(plan, positions, q, k)
        assert torch.equal(yq, want_q) and torch.equal(yk, want_k)
        tail = buf[:, 7 * 128:].clone()
        heads_first = q.transpose(0, 1).contiguous().transpose(0, 1)      # [heads][tokens] in memory
        assert torch.equal(nf4.rope_fwd(plan, positions, heads_first), want_q)
        rq, rk = nf4.rope_fwd(plan, positions, q, k, inplace=True)
        assert rq is q and torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(buf[:, 7 * 128:], tail)


def test_in_place_refuses_rows_that_share_memory():
    plan = nf4.rope_plan(64)
    positions = torch.arange(5, dtype=torch.int32, device="cuda")
    x = torch.randn((5, 4, 64), device="cuda")
    keep = x.clone()
    for bad in (x[:1].expand(5, 4, 64), x.as_strided((5, 4, 64), (128, 64, 1)), x[:, :1].expand(5, 4, 64)):
        with pytest.raises(nf4.NF4Error):
            nf4.rope_fwd(plan, positions, bad, inplace=True)
        with pytest.raises(nf4.NF4Error):
            nf4.rope_fwd(plan, positions, torch.zeros_like(x), bad, inplace=True)
    with pytest.raises(nf4.NF4Error):
        nf4.rope_fwd(plan, positions, x, x, inplace=True)
    assert torch.equal(x, keep)
    # what is only read may repeat: one head for all, one token for all, one row for both
    for one in (x[:, :1], x[:1], x[:1, :1]):
        y = nf4.rope_fwd(plan, positions, one.expand(5, 4, 64))
        assert torch.equal(y, nf4.rope_fwd(plan, positions, one.expand(5, 4, 64).contiguous()))
    y = nf4.rope_fwd(plan, positions, x[:1].expand(5, 4, 64))
    assert torch.equal(y, nf4.rope_fwd(plan, positions, x[:1].expand(5, 4, 64).contiguous()))
    heads_first = x.transpose(0, 1).contiguous().transpose(0, 1)
    want = nf4.rope_fwd(plan, positions, x)
    assert torch.equal(nf4.rope_fwd(plan, positions, heads_first, inplace=True), want) and torch.equal(heads_first, want)


def test_in_place_moves_the_version():
    plan = nf4.rope_plan(64)
    positions = torch.arange(5, dtype=torch.int32, device="cuda")
    w = torch.randn((5, 4, 64), device="cuda", requires_grad=True)
    x, k = torch.randn((5, 4, 64), device="cuda"), torch.randn((5, 2, 64), device="cuda")
    y = (w * x).sum()                         # the product's gradient needs x as it is now
    before = x._version, k._version
    nf4.rope_fwd(plan, positions, x, k)
    assert (x._version, k._version) == before
    nf4.rope_fwd(plan, positions, x, k, inplace=True)
    assert x._version > before[0] and k._version > before[1]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        z = x.clone()
        nf4.rope_fwd(plan, positions, z, inplace=True)
    nf4.rope_fwd(plan, positions, z, inplace=True)


def test_in_place_refuses_what_autograd_records():
    plan = nf4.rope_plan(64)
    positions = torch.arange(5, dtype=torch.int32, device="cuda")
    leaf, k = torch.randn((5, 4, 64), device="cuda", requires_grad=True), torch.randn((5, 2, 64), device="cuda")
    keep = leaf.detach().clone()
    for q, kk in ((leaf, None), (leaf * 1, None), (k, leaf), (leaf, k)):
        with pytest.raises(ValueError, match="in place"):
            nf4.rope_fwd(plan, positions, q, kk, inplace=True)
    assert torch.equal(leaf, keep)
    with torch.no_grad():
        nf4.rope_fwd(plan, positions, leaf, inplace=True)
    assert torch.equal(leaf, nf4.rope_fwd(plan, positions, keep))


def test_extreme_positions_values_and_nothing():
    plan = nf4.rope_plan(128)
    positions = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9], dtype=torch.int32, device="cuda")
    x = torch.randn((6, 2, 128), device="cuda")
    check(nf4.rope_fwd(plan, positions, x), x, positions, 128, False, {}, False, torch.float32)
    x[1, 0, 5], x[2, 1, 64] = float("nan"), float("inf")
    y = nf4.rope_fwd(plan, positions, x)
    # only the pairs of the odd values are touched by them
    assert int((~torch.isfinite(y)).sum()) == 4
    assert nf4.rope_fwd(plan, positions[:0], x[:0]).shape == (0, 2, 128)


def test_backward_is_the_transpose():
    # sum(w . fwd(x)) = sum(bwd(w) . x) up to fp32 rounding of 2 * 64 * 3 products
    plan = nf4.rope_plan(64, interleaved=True, **SCALED["parts"])
    x, w = torch.randn((9, 3, 96), device="cuda"), torch.randn((9, 3, 96), device="cuda")
    positions = torch.arange(9, dtype=torch.int32, device="cuda") * 1000
    a = (w.double() * nf4.rope_fwd(plan, positions, x).double()).sum()
    b = (nf4.rope_bwd(plan, positions, w).double() * x.double()).sum()
    assert abs(a - b) <= 2e-6 * float((w.abs() * x.abs()).sum() * 2)


def test_refused_tensors():
    plan = nf4.rope_plan(64)
    q = torch.zeros((4, 2, 64), device="cuda")
    p = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: nf4.rope_fwd(plan, p.long(), q), lambda: nf4.rope_fwd(plan, p, q.half()),
                lambda: nf4.rope_fwd(plan, p[:3], q), lambda: nf4.rope_fwd(plan, p, q, q.bfloat16()),
                lambda: nf4.rope_fwd(plan, p, q.transpose(1, 2)), lambda: nf4.rope_fwd(plan, p, q.cpu()),
                lambda: nf4.rope_fwd(plan, p, q[0])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nf4.NF4Error):
        nf4.rope_fwd(nf4.rope_plan(128), p, q)
