"""The norms around a block on the GPU against float64.

Bounds.  A row's sum of squares takes at most 8 x 4 + 6 + 16 additions one after the other in a thread, a wave and the
waves, each with 2^-24: 2^-18 of the factor covers half of that sum's error, the mean, the root and the
products after it.  Gradients of fp32 carry that times the sizes of the terms (step_ref gives them), sums over M tokens
(M + 64) 2^-24 of the sum of magnitudes beside it.  A store rounds by 2^-8 (bf16) or 2^-24 of the value."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import step_ref as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
UP = 2.0 ** -18


def half_step(t):
    return torch.finfo(t).eps / 2


class Case:
    def __init__(self, M, K, stream=BF16, weights=BF16, block=True, pre="weight", post="weight", gate=1, scale=0.7, eps=1e-6,
                 later=True, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed + 7 * M + K)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        near = lambda: (1 + 0.3 * rand(K)).to(weights)  # noqa: E731
        self.M, self.K, self.stream = M, K, stream
        self.h = (rand(M, K) * (0.1 + rand(M, 1).abs())).to(stream)
        self.x = (rand(M, K) * 3).to(BF16) if block else None
        self.dy = rand(M, K).to(BF16) if pre else None
        self.dh = rand(M, K).to(stream) if later else None
        kind = lambda v: near() if v == "weight" else v  # noqa: E731
        self.how = dict(pre=kind(pre), post=kind(post) if block else None, scale=scale, eps=eps,
                        gate=None if not (gate and block) else rand(gate, K).to(weights) if gate != "one" else rand(K).to(weights))

    def host(self):
        move = lambda v: v.cpu() if torch.is_tensor(v) else v  # noqa: E731
        return [move(v) for v in (self.h, self.x, self.dy, self.dh)], {k: move(v) for k, v in self.how.items()}

    def forward(self, **kw):
        return nf4.block_norm_fwd(self.h, self.x, **self.how, **kw)

    def check_forward(self):
        (h, x, _, _), how = self.host()
        new, y = self.forward()
        want, norm = ref.block_norm(h, x, **how)
        if x is None:
            assert new is self.h
        else:
            assert new.dtype == self.stream and new.is_contiguous()
            near(new, want, UP * (want - h.double()).abs() + half_step(self.stream) * want.abs() + 2.0 ** -23 * (want.abs() + h.double().abs()))
        if how["pre"] is None:
            assert y is None
        else:
            want = norm(new.cpu())
            assert y.dtype == BF16 and y.is_contiguous()
            near(y, want, (UP + half_step(BF16)) * want.abs())
        return new, y

    def backward(self, need_weights=True, **kw):
        got = nf4.block_norm_bwd(self.h, self.dy, self.dh, self.x, need_weights=need_weights, **self.how, **kw)
        return dict(zip(("dh", "dx", "dpre", "dpost", "dgate"), got))

    def check_backward(self, need_weights=True):
        (h, x, dy, dh), how = self.host()
        got = self.backward(need_weights)
        want, size = ref.block_norm_back(h, dy, dh, x, **how)
        for name, v in got.items():
            if name in ("dpre", "dpost", "dgate") and not need_weights:
                assert v is None
                continue
            assert (v is None) == (name not in want), name
            if v is None:
                continue
            step = {"dh": half_step(self.stream), "dx": half_step(BF16)}.get(name, 2.0 ** -24)
            many = (self.M + 64) * 2.0 ** -24 if name in ("dpre", "dpost", "dgate") else 0
            near(v, want[name], (UP + many) * size[name] + step * want[name].abs(), name)
        return got


def near(got, want, tol, name=""):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    assert torch.all(err <= tol + 1e-40), (name, float((err / (tol + 1e-40)).max()))


SIZES = [(1, 1), (3, 7), (5, 64), (4, 513), (33, 1000), (17, 1024), (9, 1032), (20, 2501), (6, 4096), (3, 4104), (5, 8192),
         (2, 8200), (3, 16384), (2, 20001), (1, 32768), (1, 32765), (700, 96)]


@pytest.mark.parametrize("M,K", SIZES)
@pytest.mark.parametrize("stream", [F32, BF16])
@pytest.mark.parametrize("weights", [F32, BF16])
def test_values(M, K, stream, weights):
    c = Case(M, K, stream, weights)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("M,K", [(33, 1000), (12, 2501)])
@pytest.mark.parametrize("block", [True, False])
@pytest.mark.parametrize("pre", ["weight", True, None])
@pytest.mark.parametrize("post", ["weight", True, None])
@pytest.mark.parametrize("later", [True, False])
def test_forms(M, K, block, pre, post, later):
    if not block and (pre is None or post is not None):
        pytest.skip("nothing to compute, or a block's norm without a block")
    for gate in (None, "one", 3) if block else (None,):
        c = Case(M, K, F32, F32, block, pre, post, gate, later=later)
        c.check_forward()
        c.check_backward()
        c.check_backward(need_weights=False)


@pytest.mark.parametrize("K", [40, 1000, 4100])
@pytest.mark.parametrize("M,gates", [(1, 1), (6, 6), (6, 3), (6, 2), (5000, 1), (5000, 5000), (5000, 8), (5000, 1250), (5000, 2500), (4998, 833)])
def test_gates(K, M, gates):
    # gates whose tokens lie in one worker's stretch, across several, and several to one
    if M * K > 6e6:
        M, gates = M // 2, max(1, gates // 2) if gates % 2 == 0 or gates == 1 else gates
    if M % gates:
        gates = 1
    c = Case(M, K, BF16, BF16, gate=gates)
    c.check_forward()
    c.check_backward()


@pytest.mark.parametrize("M,K,stream,weights", [(600, 8200, F32, F32), (600, 16384, BF16, BF16), (600, 9999, BF16, F32), (300, 20001, BF16, BF16),
                                                (300, 24576, F32, F32)])
def test_wide_rows_of_several_tokens_a_worker(M, K, stream, weights):
    # past a width of 8192 the sums over tokens lie elsewhere: stretches of two and three rows, gates that begin and end inside them
    for gate in (None, 1, 5, 100, M // 2, M):
        c = Case(M, K, stream, weights, gate=gate)
        c.check_backward()
        if gate in (1, 5):
            c.check_backward(need_weights=False)
    c.check_forward()
    c = Case(M, K, stream, weights, post=None, gate=M // 3)
    c.check_backward()


@pytest.mark.parametrize("stream", [F32, BF16])
@pytest.mark.parametrize("M,K", [(2100, 16384), (1030, 32768)])
def test_many_wide_rows_as_alone(M, K, stream):
    c = Case(M, K, stream, BF16)
    new, y = c.forward()
    back = c.backward()
    plain = c.backward(need_weights=False)
    assert torch.equal(plain["dh"], back["dh"]) and torch.equal(plain["dx"], back["dx"])
    for row in (0, 1, M // 2, M - 1):
        one = slice(row, row + 1)
        t, z = nf4.block_norm_fwd(c.h[one], c.x[one], **c.how)
        assert torch.equal(new[one], t) and torch.equal(y[one], z)
        got = nf4.block_norm_bwd(c.h[one], c.dy[one], c.dh[one], c.x[one], **c.how)
        assert torch.equal(back["dh"][one], got[0]) and torch.equal(back["dx"][one], got[1])
    want, size = 0, 0
    for a in range(0, M, 100):
        h, t = c.h[a:a + 100].double(), c.dy[a:a + 100].double()
        term = t * h / (h.square().mean(1, keepdim=True) + c.how["eps"]).sqrt()
        want, size = want + term.cumsum(0)[-1], size + term.abs().cumsum(0)[-1]
    near(back["dpre"], want.cpu(), (UP + (M + 64) * 2.0 ** -24) * size.cpu() + 2.0 ** -24 * want.abs().cpu())


def test_strides_and_alignment():
    for pad, first in ((0, 0), (3, 1), (8, 8)):
        c, d = (Case(11, 1003, BF16, F32, gate=11) for _ in range(2))
        for name in ("h", "x", "dy", "dh"):
            buf = torch.full((11, 1003 + pad + first), float("nan"), dtype=getattr(c, name).dtype, device="cuda")
            view = buf[:, first:first + 1003]
            view.copy_(getattr(c, name))
            setattr(d, name, view)
        for a, b in zip(c.forward(), d.forward()):
            assert torch.equal(a, b)
        for a, b in zip(c.backward().values(), d.backward().values()):
            assert torch.equal(a, b)
    # one row for all tokens
    c = Case(9, 200, BF16, F32)
    d = Case(9, 200, BF16, F32)
    c.x = c.x[:1].repeat(9, 1)
    d.x = c.x[:1].expand(9, 200)
    assert torch.equal(c.forward()[0], d.forward()[0])


def test_in_place():
    c = Case(7, 513)
    want, y = c.forward()
    version, buf = c.h._version, torch.zeros((7, 600), dtype=BF16, device="cuda")
    buf[:, 5:518] = c.h
    got, z = nf4.block_norm_fwd(c.h, c.x, inplace=True, **c.how)
    assert got is c.h and torch.equal(got, want) and torch.equal(z, y) and c.h._version > version
    view = buf[:, 5:518]
    nf4.block_norm_fwd(view, c.x, inplace=True, **c.how)
    assert torch.equal(view, want) and not buf[:, :5].any() and not buf[:, 518:].any()
    for bad in (c.h[:1].expand(7, 513), c.h.flatten()[:7 * 100 + 513].as_strided((7, 513), (100, 1))):
        with pytest.raises(nf4.NF4Error):
            nf4.block_norm_fwd(bad, c.x, inplace=True, **c.how)
    leaf = c.h.float().requires_grad_(True)
    with pytest.raises(ValueError):
        nf4.block_norm_fwd(leaf, c.x, inplace=True, **c.how)


@pytest.mark.parametrize("K", [200, 2500, 20000])
def test_squares_past_fp32(K):
    # values whose squares overflow, or vanish: the norm is that of the scaled row
    c = Case(4, K, F32, F32, gate=None, scale=1.0, post="weight")
    c.h = c.h * torch.tensor([1e37, 1e-30, 3e18, 1.0], device="cuda")[:, None]
    c.x = (c.x.float() * torch.tensor([1.0, 1e-25, 1e25, 3e30], device="cuda")[:, None]).to(BF16)
    c.check_forward()
    c.h = c.h * torch.tensor([1.0, 1.0, 1e5, 1.0], device="cuda")[:, None]
    c.check_backward()


def test_rows_of_nothing_and_of_the_non_finite():
    c = Case(5, 1000, F32, F32)
    clean = c.forward(), c.backward()
    c.h, c.x = c.h.clone(), c.x.clone()
    c.h[1], c.x[1] = 0, 0
    c.x[3, 17] = float("inf")
    c.h[4, 3] = float("nan")
    new, y = c.forward()
    assert not new[1].any() and not y[1].any()
    assert torch.isnan(new[3, 17]) and torch.isnan(new[4, 3]) and torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    assert torch.equal(new[0], clean[0][0][0]) and torch.equal(y[2], clean[0][1][2])
    back = c.backward()
    assert torch.isfinite(back["dh"][:4]).all() and torch.isnan(back["dh"][4]).any()
    assert torch.equal(back["dh"][0], clean[1]["dh"][0]) and torch.equal(back["dx"][2], clean[1]["dx"][2])


def test_offsets_past_32_bits():
    # rows beyond 2^32 bytes of every operand, against the same rows alone
    M, K = 140000, 16384
    g = torch.Generator(device="cuda").manual_seed(1)
    h = torch.empty((M, K), dtype=BF16, device="cuda")
    for a in range(0, M, 10000):
        h[a:a + 10000] = torch.randn((10000, K), generator=g, device="cuda")
    gate = torch.rand((2, K), generator=g, device="cuda").to(BF16)
    s, y = nf4.block_norm_fwd(h, h, gate=gate)
    dh, dx, _, _, dgate = nf4.block_norm_bwd(s, y, None, h, gate=gate)
    for row in (0, M // 2 - 1, M // 2, M - 1):
        one = slice(row, row + 1)
        own = gate[row // (M // 2)]
        t, z = nf4.block_norm_fwd(h[one], h[one], gate=own)
        assert torch.equal(s[one], t) and torch.equal(y[one], z)
        back = nf4.block_norm_bwd(t, z, None, h[one], gate=own)
        assert torch.equal(dh[one], back[0]) and torch.equal(dx[one], back[1])
    # each half's gate has the sum of its own tokens: the two of one kind of rows, as large within its spread
    assert torch.isfinite(dgate).all() and dgate.shape == (2, K)
    part = sum((h[a:a + 10000].float() * dh[a:a + 10000].float()).double().sum(0) for a in range(0, M // 2, 10000))
    assert float((dgate[0].double() - part).norm()) <= 0.02 * float(part.norm())


def test_no_tokens():
    c = Case(0, 64, gate=1)
    new, y = c.forward()
    assert new.shape == y.shape == (0, 64)
    got = c.backward()
    assert got["dh"].shape == got["dx"].shape == (0, 64)
    assert not got["dpre"].any() and not got["dpost"].any() and not got["dgate"].any() and got["dgate"].shape == (1, 64)


def test_repeats_bit_for_bit_on_any_stream():
    c = Case(1500, 1000, gate=5)
    a = c.backward()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        b = c.backward()
        f = c.forward()
    torch.cuda.current_stream().wait_stream(other)
    assert all(torch.equal(a[k], b[k]) for k in a)
    assert all(torch.equal(u, v) for u, v in zip(c.forward(), f))


def test_refusals():
    c = Case(6, 64)
    w = c.how
    bad = [dict(gate=torch.ones((4, 64), device="cuda", dtype=BF16)), dict(gate=torch.ones((2, 63), device="cuda", dtype=BF16)),
           dict(pre=torch.ones(63, device="cuda", dtype=BF16)), dict(pre=torch.ones(64, device="cuda")),       # two types of weights
           dict(post=torch.ones(64, dtype=BF16)), dict(pre=torch.ones(64, device="cuda", dtype=torch.float16))]
    for b in bad:
        with pytest.raises(ValueError):
            nf4.block_norm_fwd(c.h, c.x, **{**w, **b})
    for b in (dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf"))):
        with pytest.raises(nf4.NF4Error):
            nf4.block_norm_fwd(c.h, c.x, **{**w, **b})
    for h, x in ((c.h.half(), c.x), (c.h.cpu(), c.x), (c.h, c.x.float()), (c.h, c.x[:5]), (c.h[0], c.x), (c.h.t(), c.x.t()), (c.h, c.x.cpu())):
        with pytest.raises(ValueError):
            nf4.block_norm_fwd(h, x, **w)
    with pytest.raises(nf4.NF4Error):
        nf4.block_norm_fwd(c.h, None, pre=None)
    with pytest.raises(nf4.NF4Error):
        nf4.block_norm_fwd(c.h, None, post=w["post"])
    with pytest.raises(nf4.NF4Error):
        nf4.block_norm_fwd(torch.zeros((1, 32769), device="cuda"))
    with pytest.raises(ValueError):
        nf4.block_norm_bwd(c.h, None, c.dh, c.x, **w)
    with pytest.raises(ValueError):
        nf4.block_norm_bwd(c.h, c.dy, c.dh.float(), c.x, **w)
    with pytest.raises(TypeError):
        nf4.block_norm_fwd(np.zeros((6, 64)), c.x)
