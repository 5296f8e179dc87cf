"""Penalties, biases and masks of logits on the GPU against float64.

Bounds.  Four fp32 operations at most, each within 2^-24 of the sizes that meet in it: 2^-22 of them, and the store's
rounding, 2^-24 or 2^-8 (bf16) of the value."""
import math

import numpy as np
import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import step_ref as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def cuda(x, dtype=torch.int32):
    return None if x is None else torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def words(R, V, seed, share=0.5):
    r = np.random.RandomState(seed)
    bits = r.rand(R, (V + 31) // 32 * 32) < share
    w = (bits.reshape(R, -1, 32) * (1 << np.arange(32, dtype=np.int64))).sum(-1)
    return np.where(w >= 1 << 31, w - (1 << 32), w)


class Case:
    def __init__(self, R, V, dtype=F32, history=0, biases=0, grammar=False, each=False, seed=0, one=False):
        r = np.random.RandomState(seed + R + V)
        self.z = torch.tensor(r.randn(R, V) * 3, dtype=torch.float32).to(dtype).cuda()
        n = 1 if one else R
        self.kw = {}
        if history:
            self.kw["history"] = (r.rand(n, history) ** 3 * V * 1.02).astype(np.int64) - 1       # some outside
            self.kw["lengths"] = r.randint(-1, history + 2, R)
            self.kw["prompts"] = r.randint(-1, history + 2, R)
            number = lambda lo, hi: (lo + (hi - lo) * r.rand(R)).astype(np.float32) if each else float(np.float32(lo + (hi - lo) * r.rand()))  # noqa: E731
            self.kw.update(repetition=number(0.8, 1.5), presence=number(-0.2, 1), frequency=number(-0.1, 0.3))
        if biases:
            self.kw["bias_ids"] = r.randint(-1, V + 1, (n, biases))
            self.kw["bias"] = (r.randn(n, biases) * 5).astype(np.float32)
        if grammar:
            self.kw["allowed"] = words(n, V, seed)

    def device(self):
        f = {"bias", "repetition", "presence", "frequency"}
        return {k: v if np.ndim(v) == 0 else cuda(v, F32 if k in f else torch.int32) for k, v in self.kw.items()}

    def check(self):
        got = nf4.shape_logits(self.z, **self.device())
        want, size = ref.shape_logits(self.z.float().cpu().numpy(), **self.kw)
        step = 2.0 ** -22 * size + (2.0 ** -8 if self.z.dtype == BF16 else 0) * np.abs(np.where(np.isinf(want), 0, want))
        y = got.float().cpu().numpy().astype(np.float64)
        assert got.dtype == self.z.dtype and got.is_contiguous() and np.array_equal(np.isinf(y), np.isinf(want))
        ok = np.isfinite(want)
        assert np.all(np.abs(y[ok] - want[ok]) <= step[ok])
        return got


SIZES = [(1, 1), (1, 7), (3, 33), (2, 2047), (2, 2049), (5, 8193), (1, 32000), (40, 1001)]


@pytest.mark.parametrize("R,V", SIZES)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("history", [0, 1, 300])
@pytest.mark.parametrize("biases", [0, 40])
@pytest.mark.parametrize("grammar", [False, True])
def test_values(R, V, dtype, history, biases, grammar):
    Case(R, V, dtype, history, biases, grammar).check()
    Case(R, V, dtype, history, biases, grammar, each=True, one=True).check()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_batches(dtype):
    Case(70, 32001, dtype, 500, 30, True, each=True).check()
    Case(300, 9000, dtype, 3, 0, False).check()


def test_long_histories():
    Case(3, 50, history=20000).check()                              # counts of some hundreds
    Case(1, 40000, history=50000, each=True).check()
    Case(2, 30001, history=2000, biases=500, grammar=True).check()
    Case(2, 20001, history=40000, biases=70, grammar=True, each=True).check()
    Case(2, 3000, history=5, biases=70000).check()                   # more biases than tokens


@pytest.mark.parametrize("width", [1000, 32767, 32768, 70000])
def test_one_token_alone(width):
    # every count there is, beside the last entry of the biases
    z = torch.zeros((1, 3), device="cuda")
    history = torch.ones((1, width), dtype=torch.int32, device="cuda")
    ids = torch.ones((1, 65535), dtype=torch.int32, device="cuda")
    for count in (65535, 100):
        got = nf4.shape_logits(z, history, frequency=2.0, presence=0.5, bias_ids=ids[:, :count], bias=torch.arange(count, device="cuda")[None].float())
        assert got.tolist() == [[0.0, count - 1 - 2.0 * width - 0.5, 0.0]]
    got = nf4.shape_logits(z - 1, history, prompts=torch.tensor([width], dtype=torch.int32, device="cuda"), repetition=3.0, frequency=2.0)
    assert got.tolist() == [[-1.0, -3.0, -1.0]]


def test_offsets_past_32_bits():
    R, V = 18000, 128256
    z = torch.empty((R, V), dtype=BF16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for a in range(0, R, 2000):
        z[a:a + 2000] = torch.randn((2000, V), generator=g, device="cuda")
    history = torch.randint(0, V, (R, 20), generator=g, dtype=torch.int32, device="cuda")
    got = nf4.shape_logits(z, history, presence=1.0, repetition=1.5)
    for row in (0, R // 2, R - 1):
        one = slice(row, row + 1)
        assert torch.equal(got[one], nf4.shape_logits(z[one], history[one], presence=1.0, repetition=1.5))
        assert int((got[one] != z[one]).sum()) >= 15


def test_many_rows():
    z = torch.randn((70000, 3), device="cuda")
    history = torch.randint(0, 3, (70000, 2), dtype=torch.int32, device="cuda")
    got = nf4.shape_logits(z, history, presence=10.0)
    seen = torch.zeros_like(z).scatter_(1, history.long(), 1.0)
    assert torch.equal(got, z - 10 * seen)


def test_the_last_of_equal_ids_counts():
    z = torch.zeros((1, 5000), device="cuda")
    ids = [[7] * 999 + [9, 7, 4000]]
    bias = [list(range(1, 1000)) + [5, -3, 2]]
    got = nf4.shape_logits(z, bias_ids=cuda(ids), bias=cuda(bias, F32))
    assert float(got[0, 7]) == -3 and float(got[0, 9]) == 5 and float(got[0, 4000]) == 2 and int((got != 0).sum()) == 3


def test_rows_that_may_not_go_on_and_the_non_finite():
    z = torch.tensor([[math.inf, -math.inf, math.nan, 1.0, -1.0]] * 3, device="cuda")
    allowed = cuda([[0], [0b11010], [-1]])
    history = cuda([[0, 1, 2, 3, 4]] * 3)
    got = nf4.shape_logits(z, history, repetition=2.0, allowed=allowed)
    assert torch.equal(got[0], torch.full((5,), -math.inf, device="cuda"))
    assert torch.equal(got[1], torch.tensor([-math.inf, -math.inf, -math.inf, 0.5, -2.0], device="cuda"))
    assert math.isinf(got[2, 0]) and got[2, 1] == -math.inf and torch.isnan(got[2, 2]) and got[2, 3] == 0.5


def test_ids_at_the_ends():
    z = torch.ones((1, 3000), device="cuda")
    ends = [[-2 ** 31, 2 ** 31 - 1, -1, 3000, 2999, 0]]
    got = nf4.shape_logits(z, cuda(ends), presence=2.0, bias_ids=cuda(ends), bias=torch.full((1, 6), 0.5, device="cuda"))
    assert int((got != 1).sum()) == 2 and got[0, 0] == -0.5 and got[0, 2999] == -0.5


def test_strides_and_in_place():
    c = Case(6, 1001, BF16, 50, 5, True)
    want, kw = c.check(), c.device()
    buf = torch.full((6, 1100), 9.0, dtype=BF16, device="cuda")
    view = buf[:, 3:1004]
    view.copy_(c.z)
    wide = torch.zeros((6, 77), dtype=torch.int32, device="cuda")
    wide[:, 10:60] = kw["history"]
    assert torch.equal(nf4.shape_logits(view, **{**kw, "history": wide[:, 10:60]}), want)
    version = buf._version
    got = nf4.shape_logits(view, inplace=True, **kw)
    assert got is view and torch.equal(view, want) and buf._version > version
    assert torch.all(buf[:, :3] == 9) and torch.all(buf[:, 1004:] == 9)
    one = c.z[:1].expand(6, 1001)
    assert torch.equal(nf4.shape_logits(one, **kw), nf4.shape_logits(one.contiguous(), **kw))
    for bad in (one, buf.flatten().as_strided((6, 1001), (500, 1))):
        with pytest.raises(nf4.NF4Error):
            nf4.shape_logits(bad, inplace=True, **kw)
    with pytest.raises(ValueError):
        nf4.shape_logits(c.z.clone().requires_grad_(True), inplace=True, **kw)


def test_nothing_to_do():
    z = torch.randn((3, 100), device="cuda")
    none = torch.empty((3, 0), dtype=torch.int32, device="cuda")
    assert torch.equal(nf4.shape_logits(z), z)
    assert torch.equal(nf4.shape_logits(z, none, presence=3.0, bias_ids=none, bias=none.float()), z)
    assert nf4.shape_logits(z[:0]).shape == (0, 100)


def test_refusals():
    z = torch.randn((3, 100), device="cuda")
    ids = torch.zeros((3, 4), dtype=torch.int32, device="cuda")
    for bad in (dict(history=ids.long()), dict(history=ids[:2]), dict(history=ids[0]), dict(history=ids.cpu()), dict(lengths=ids[:, 0]),
                dict(history=ids, lengths=ids[0]), dict(history=ids, prompts=ids[:, 0].long()), dict(bias_ids=ids), dict(bias=ids.float()),
                dict(bias_ids=ids, bias=ids), dict(bias_ids=ids, bias=ids[:, :3].float()), dict(allowed=ids[:, :3]), dict(allowed=ids.bool()),
                dict(history=ids, repetition=torch.ones(2, device="cuda")), dict(history=ids, presence=torch.ones(3)), dict(history=ids.t())):
        with pytest.raises(ValueError):
            nf4.shape_logits(z, **bad)
    for bad in (dict(history=ids, repetition=0.0), dict(history=ids, repetition=-1.0), dict(history=ids, presence=float("nan"))):
        with pytest.raises(nf4.NF4Error):
            nf4.shape_logits(z, **bad)
    for bad in (z.half(), z.cpu(), z[0], z.t()):
        with pytest.raises(ValueError):
            nf4.shape_logits(bad)
