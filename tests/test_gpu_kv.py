"""The paged 8-bit cache on the GPU against float64: appends and attention.

Bounds.  Append: scales are exact; a code is within half a step of the exact quotient (2^-4 of
it, or 2^-10 among the subnormals) but for the fp32 rotation's 1e-6 of the pair.  Attention:
scores carry fp32 rounding, at most D 2^-24 sum|q k| scale (below 2^-13 of a weight for the
sizes here), weights 2^-12 as fp16, outputs 2^-8 of themselves as bf16: 2^-8 |o| + 2^-10 max|v|."""
import ctypes
import math

import numpy as np
import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import decoder_abi as dec
import decoder_ref as ref

pytestmark = pytest.mark.gpu


def dev(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


class Case:
    """Sequences with `lengths` tokens before and `counts` new ones, on pages dealt out in no order."""

    def __init__(self, lengths, counts, page=16, kv=2, heads=4, dim=128, seed=0, spare=3, fill=True):
        r = np.random.RandomState(seed)
        self.page, self.kv, self.heads, self.dim = page, kv, heads, dim
        self.lengths, self.counts = np.array(lengths), np.array(counts)
        self.starts = np.concatenate([[0], np.cumsum(counts)])
        need = [max(0, -(-max(0, n + c) // page)) for n, c in zip(lengths, counts)]
        total = sum(need) + spare
        order = r.permutation(total)
        self.table = np.full((len(need), max(need + [1])), -1, np.int64)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.tokens = int(self.starts[-1])
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.cache = nf4.kv_cache(total, kv, dim, page)
        if fill:
            # codes of every finite value, scales of several sizes
            self.cache.codes.copy_((rand(total, 2, kv, page, dim) * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
            self.cache.scales.copy_(torch.exp2(torch.randint(-7, -3, (total, 2, kv), generator=g, device="cuda").float()))
        qkv = rand(self.tokens, heads + 2 * kv, dim).bfloat16()
        self.q, self.k, self.v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]

    def meta(self):
        return dev(self.starts), dev(self.lengths), dev(self.table)

    def host(self):
        return self.cache.codes.cpu().numpy(), self.cache.scales.cpu().numpy()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_append(c, rope=None, plan=None, with_q=True):
    codes0, scales0 = c.host()
    want, scales, quotient = ref.append(codes0, scales0, f64(c.k), f64(c.v), c.starts, c.lengths, c.table, rope)
    q = nf4.kv_append(c.cache, c.k, c.v, *c.meta(), rope=plan, q=c.q if with_q else None)
    codes, got_scales = c.host()
    assert np.array_equal(got_scales, scales)
    new = ~np.isnan(quotient)
    assert np.array_equal(codes[~new], want[~new])                  # what was there, written again or not
    value = ref.e4m3_values()
    x, y = quotient[new], value[codes[new]]
    nan = np.isnan(value[want[new]])
    assert np.array_equal(np.isnan(y), nan)
    step = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -10)
    assert np.all(np.abs(y - x)[~nan] <= (step + 1e-6 * 640)[~nan])
    # nearly all codes are the nearest to the exact quotient (rounding moves one in some 10^4 across a tie)
    assert np.mean(codes[new] != want[new]) <= 1e-3
    if plan is None:
        assert np.array_equal(codes, want)
    return q


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("rotary,inter", [(None, False), (1.0, False), (1.0, True), (0.5, True), (22, False)])
def test_append(dim, page, rotary, inter):
    for lengths, counts, kv, heads in (([0], [1], 1, 1), ([5, 0, 63, 129], [1, 1, 1, 1], 3, 6),
                                       ([0, 17, 100, 0, 250, 31], [40, 3, 0, 300, 7, 1], 5, 10)):
        c = Case(lengths, counts, page=page, kv=kv, heads=heads, dim=dim, seed=dim + page + kv)
        plan = rope = None
        if rotary is not None:
            n = rotary if rotary == 22 else int(dim * rotary)
            plan = nf4.rope_plan(n, interleaved=inter, scaling="parts", factor=4.0, original_length=128)
            theta, mag = ref.theta_of(n, scaling="parts", factor=4.0, original_length=128)
            rope = (n, inter, theta, mag)
        q = check_append(c, rope, plan)
        positions = dev(np.concatenate([np.arange(n, n + k) for n, k in zip(lengths, counts)]))
        want = nf4.rope_fwd(plan, positions, c.q) if plan else c.q
        assert torch.equal(q, want)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_one_head_for_all(dim):
    # keys, values and queries whose heads are one: an expanded tensor, as its copies
    plan = nf4.rope_plan(dim)
    c, d = (Case([5, 0, 40], [3, 20, 1], page=16, kv=3, heads=6, dim=dim, seed=23) for _ in range(2))
    q, k, v = (x[:, :1].contiguous() for x in (c.q, c.k, c.v))
    a = nf4.kv_append(c.cache, k.expand(-1, 3, -1), v.expand(-1, 3, -1), *c.meta(), rope=plan, q=q.expand(-1, 6, -1))
    b = nf4.kv_append(d.cache, k.repeat(1, 3, 1), v.repeat(1, 3, 1), *d.meta(), rope=plan, q=q.repeat(1, 6, 1))
    assert torch.equal(a, b) and torch.equal(c.cache.codes, d.cache.codes) and torch.equal(c.cache.scales, d.cache.scales)
    assert torch.equal(nf4.kv_attention(c.cache, a[:, :1].expand(-1, 6, -1), *c.meta()),
                       nf4.kv_attention(d.cache, a[:, :1].repeat(1, 6, 1), *d.meta()))


def test_append_moves_the_versions():
    c = Case([5, 0], [3, 1], page=16, kv=2, heads=4, dim=64, seed=24)
    before = c.cache.codes._version, c.cache.scales._version, c.q._version
    q = nf4.kv_append(c.cache, c.k, c.v, *c.meta(), q=c.q)
    assert c.cache.codes._version > before[0] and c.cache.scales._version > before[1] and c.q._version == before[2]
    keep = c.cache.codes._version
    nf4.kv_attention(c.cache, q, *c.meta())
    assert c.cache.codes._version == keep


def test_append_many_sequences():
    r = np.random.RandomState(1)
    check_append(Case(r.randint(0, 90, 300), r.randint(0, 4, 300), page=32, kv=2, dim=64, seed=4), with_q=False)
    check_append(Case(r.randint(0, 9, 4200), np.ones(4200, int), page=16, kv=1, heads=1, dim=64, seed=5))


def test_append_scale_boundaries_and_growth():
    c = Case([0, 3], [1, 1], page=16, kv=1, heads=1, dim=64, seed=2)
    c.k, c.v = torch.zeros_like(c.k), torch.zeros_like(c.v)
    c.v[0, 0, 0], c.v[1, 0, 63] = 448.0, -450.0                    # exactly the largest code; just past it
    c.k[1, 0, 7] = 3.0e38                                            # past every scale: clamped at 448 * 2^50
    check_append(c)
    page = c.table[1, 0]
    assert float(c.cache.scales[c.table[0, 0], 1, 0]) == 1.0 and float(c.cache.scales[page, 1, 0]) == 2.0
    assert float(c.cache.scales[page, 0, 0]) == 2.0 ** 50 and int(c.cache.codes[page, 0, 0, 3, 7]) == 126
    # nothing but zeros on a fresh page: the smallest scale
    assert float(c.cache.scales[c.table[0, 0], 0, 0]) == 2.0 ** -50


def test_append_non_finite_tokens():
    c = Case([0, 10], [20, 2], page=16, kv=3, heads=3, dim=128, seed=3)
    c.k, c.v = c.k.clone(), c.v.clone()
    c.k[4, 1, 100], c.v[17, 0, 3], c.v[20, 2, 0] = float("nan"), float("inf"), -float("inf")
    c.k[:16, 2], c.v[:16, 2] = float("nan"), 0                       # a page with no finite token
    plan = nf4.rope_plan(128)
    check_append(c, (128, False, *ref.theta_of(128)), plan)
    out = nf4.kv_attention(c.cache, c.q, *c.meta())
    bad = torch.zeros((22, 3), dtype=torch.bool)
    bad[4:20, 1] = bad[17:20, 0] = bad[20:, 2] = bad[:20, 2] = True
    assert torch.equal(torch.isnan(out).all(-1).cpu(), bad) and torch.equal(torch.isnan(out).any(-1).cpu(), bad)


def test_append_unused_rows_and_absent_pages():
    c = Case([-1, 30, -5, 20], [1, 4, 8, 2], page=16, kv=2, heads=2, dim=64, seed=6)
    c.table[1, 2:] = -1                                              # positions 32, 33 have no page
    c.table[3, 1] = 10 ** 6
    before = c.cache.codes.clone()
    check_append(c, with_q=False)
    changed = (c.cache.codes != before).flatten(1).any(1).sum()
    assert int(changed) <= 2                                         # one page of sequence 1, one of sequence 2


def check_attention(c, scale=None, **kw):
    codes, scales = c.host()
    out = nf4.kv_attention(c.cache, c.q, *c.meta(), scale=scale, **kw)
    want, reach = ref.attention(codes, scales, f64(c.q), c.starts, c.lengths, c.table, scale or 1 / math.sqrt(c.dim))
    got = f64(out)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * reach[..., None]), (err / (reach[..., None] + 1e-30)).max()
    return out


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("kv,heads", [(1, 1), (2, 2), (2, 14), (1, 40), (3, 48)])
def test_attention_single_tokens(dim, page, kv, heads):
    c = Case([0, 1, 14, 15, 16, 31, 32, 127, 128, 300, 777], [1] * 11, page=page, kv=kv, heads=heads, dim=dim, seed=dim + heads)
    check_attention(c, max_new=1, max_length=778)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,heads", [(2, 2), (1, 5), (2, 32)])
def test_attention_chunks(dim, kv, heads):
    c = Case([0, 100, 0, 45, 3, 260], [1, 33, 130, 0, 17, 64], page=32, kv=kv, heads=heads, dim=dim, seed=dim + heads)
    a = check_attention(c, max_new=130, max_length=330)
    # sizes that the launch was not told, or told too large, change nothing but the order of sums
    for kw in (dict(max_new=1, max_length=1), dict(max_new=4000, max_length=100000), {}):
        b = nf4.kv_attention(c.cache, c.q, *c.meta(), **kw)
        assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -10 * 8)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,heads", [(1, 2), (2, 16)])
def test_attention_few_tokens_behind_many_keys(dim, kv, heads):
    # short chunks, and sequences of a few rows among longer ones; then with a kernel for each kind
    c = Case([1500, 900, 3, 1111, 700], [33, 20, 40, 1, 0], page=64, kv=kv, heads=heads, dim=dim, seed=dim + kv)
    check_attention(c, max_new=40, max_length=1533)
    check_attention(c, max_new=40, max_length=200000)


@pytest.mark.parametrize("dim,page,counts", [(128, 64, [300, 290, 45, 0]), (64, 16, [310, 200, 90, 3]), (64, 32, [500, 333, 270, 1]),
                                             (128, 16, [400, 300, 350, 40]), (256, 128, [70, 200, 1, 100])])
def test_attention_many_blocks(dim, page, counts):
    # more waves than run at once: blocks of several sequences in the order of their keys, alone and two to a block
    check_attention(Case([150, 10, 400, 33], counts, page=page, kv=2, heads=64, dim=dim, seed=sum(counts)), max_new=max(counts), max_length=550)


@pytest.mark.parametrize("kv,heads", [(8, 8), (8, 64)])
def test_attention_with_a_capacity_for_max_new(kv, heads):
    # single tokens, and a stated maximum far past them, as of a server's fixed limits
    c = Case([300, 7, 64, 1000, 0, 511, 33, 100], [1] * 8, page=64, kv=kv, heads=heads, dim=128, seed=kv + heads)
    a = check_attention(c, max_new=1, max_length=1024)
    for new in (8, 4096, 1 << 20, (1 << 23) - 1):
        b = check_attention(c, max_new=new, max_length=1 << 20)
        assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -10 * 8)


def test_attention_long_split():
    c = Case([40000, 3, 20011], [1, 1, 2], page=64, kv=1, heads=4, dim=128, seed=9)
    check_attention(c, max_new=2, max_length=40001)


@pytest.mark.parametrize("counts", [[300, 200], [3, 1]])
def test_attention_long_reach(counts):
    # a table of 2^25 positions, nearly all of them absent: with and without a stated length
    c = Case([0, 100], counts, page=256, kv=4, heads=32, dim=64, seed=21)
    c.table = np.concatenate([c.table, np.full((2, (1 << 25) // 256 - c.table.shape[1]), -1)], axis=1)
    a = check_attention(c)
    b = check_attention(c, max_new=max(counts), max_length=300)
    assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -10 * 8)
    check_attention(c, max_length=2 ** 31 - 1)


def test_attention_sharp_and_flat_scores():
    c = Case([500, 500], [1, 1], page=16, kv=2, heads=4, dim=64, seed=11)
    c.q = c.q * 30                                                   # scores of some hundreds: one key wins
    check_attention(c, scale=1.0, max_new=1, max_length=501)
    c.q = c.q * 0
    check_attention(c, max_new=1, max_length=501)


def test_attention_zero_and_negative_scale():
    c = Case([300, 20], [1, 40], page=16, kv=2, heads=4, dim=64, seed=18)
    codes, scales = c.host()
    for scale in (-0.2, 1e-300):             # the second is zero as fp32: every key that is seen weighs the same
        want, reach = ref.attention(codes, scales, f64(c.q), c.starts, c.lengths, c.table, scale)
        got = f64(nf4.kv_attention(c.cache, c.q, *c.meta(), scale=scale))
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * reach[..., None])


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("counts", [[1], [40]])
@pytest.mark.parametrize("top", [2.0 ** 109, 2.0 ** 110, 1.9 * 2.0 ** 110])
def test_attention_of_large_queries(dim, counts, top):
    # queries near the limit where sums of 256 products with codes of 448 leave fp32, over keys of 2^-45: scores of order 1
    c = Case([300], counts, page=16, kv=2, heads=4, dim=dim, seed=dim)
    c.cache.scales[:, 0] = 2.0 ** -50
    q = c.q.float()
    c.q = (q / q.abs().amax(-1, keepdim=True) * top).bfloat16()
    check_attention(c, scale=2.0 ** 45 / top / math.sqrt(dim))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("counts", [[1], [40], [300]])
@pytest.mark.parametrize("size,scale", [(1e-28, None), (1e-38, None), (1e-7, 0.0), (1.0, 1e-300), (1e-7, 1e-30), (1.0, 1e38)])
def test_attention_factors_at_the_ends(dim, counts, size, scale):
    # keys of nothing on pages of the smallest scale, tiny queries, scales of zero, of zero as fp32 and of 2^126: every
    # key that is seen weighs the same, and none that is not
    c = Case([300], counts, page=16, kv=2, heads=4, dim=dim, seed=dim)
    c.cache.codes[:, 0] = 0
    c.cache.scales[:, 0] = 2.0 ** -50
    c.q = (c.q.float() * size).bfloat16()
    check_attention(c, scale=scale)


def test_attention_scales_far_apart():
    c = Case([600], [1], page=16, kv=1, heads=2, dim=64, seed=12)
    r = np.random.RandomState(5)
    c.cache.scales[:, 1] = dev(2.0 ** r.randint(-50, 51, (c.cache.scales.shape[0], 1)), torch.float32)
    c.cache.scales[:, 0] = 2.0 ** -9
    check_attention(c, max_new=1, max_length=601)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("counts", [[1, 1], [40, 1]])
@pytest.mark.parametrize("odd", [-math.inf, math.inf, math.nan])
def test_attention_of_non_finite_queries(dim, counts, odd):
    # keys of ones: an infinity makes every score the same one.  Such rows are NaN, others untouched
    c = Case([30, 77], counts, page=16, kv=1, heads=2, dim=dim, seed=dim)
    c.cache.codes[:, 0] = 0x38
    clean = nf4.kv_attention(c.cache, c.q, *c.meta())
    c.q = c.q.clone()
    c.q[-1, 0, dim - 1] = c.q[:-1, 1, 3] = odd
    out = nf4.kv_attention(c.cache, c.q, *c.meta())
    assert torch.isnan(out[-1, 0]).all() and torch.isnan(out[:-1, 1]).all()
    assert torch.equal(out[-1, 1], clean[-1, 1]) and torch.equal(out[:-1, 0], clean[:-1, 0])


def test_attention_hides_what_is_not_there():
    # NaN codes past the end of a sequence, on spare pages and in later tokens' keys
    c = Case([20, 5], [6, 1], page=16, kv=1, heads=2, dim=128, seed=13)
    clean = nf4.kv_attention(c.cache, c.q, *c.meta())
    for b, n in ((0, 26), (1, 6)):
        last = c.table[b, n // 16]
        c.cache.codes[last, :, :, n % 16:] = 127
    spare = sorted(set(range(c.cache.codes.shape[0])) - set(c.table[c.table >= 0].tolist()))
    c.cache.codes[spare] = 127
    c.cache.scales[spare] = float("nan")
    assert torch.equal(nf4.kv_attention(c.cache, c.q, *c.meta()), clean)
    c.cache.codes[c.table[0, 1], 0, :, 25 - 16] = 127                # the last token's key
    out = nf4.kv_attention(c.cache, c.q, *c.meta())
    assert torch.isnan(out[5]).all() and torch.equal(out[:5], clean[:5]) and torch.equal(out[6], clean[6])


def test_attention_rows_that_see_nothing():
    c = Case([-1, 4, -3, 10], [1, 1, 5, 1], page=16, kv=2, heads=6, dim=64, seed=14)
    out = check_attention(c, max_new=5, max_length=11)
    assert not out[0].any() and not out[2:5].any() and out[1].any() and out[5].any()
    c.table[1, 0] = -1                                               # no page at all
    assert not check_attention(c, max_new=5, max_length=11)[1].any()
    c.lengths[3] = 16                                                # past the table
    assert not check_attention(c, max_new=5, max_length=17)[7].any()


@pytest.mark.parametrize("dim,heads,tokens", [(128, 4, 6), (128, 16, 70), (64, 32, 70), (256, 8, 40)])
@pytest.mark.parametrize("wrong", [[2 ** 31 - 1, 2 ** 31 - 1], [-7, 10 ** 6], [-2 ** 31, -1], [3, 2]])
def test_attention_and_append_of_wrong_starts(dim, heads, tokens, wrong):
    # the first sequence is in order, the starts behind it are not: nothing but the batch's own rows is written
    c = Case([50, 20, 9], [tokens - 2, 1, 1], page=16, kv=2, heads=heads, dim=dim, seed=20)
    want = nf4.kv_attention(c.cache, c.q, *c.meta(), max_new=tokens)
    c.starts[2:] = wrong
    starts, lengths, table = c.meta()
    room = torch.full((tokens + 64, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    view = lambda x, n: dec._Heads(x.data_ptr(), n * dim, dim, n)  # noqa: E731
    q = c.q.contiguous()
    cache = dec._Cache(c.cache.codes.data_ptr(), c.cache.scales.data_ptr(), c.cache.codes.shape[0], 2, 16, dim)
    batch = dec._Batch(starts.data_ptr(), lengths.data_ptr(), table.data_ptr(), table.shape[1], tokens, 3, table.shape[1])
    by = ctypes.byref
    for length in (100, 200000):
        size = dec._library().qlora_kv_attention_workspace_bytes(by(cache), by(batch), heads, tokens, length)
        ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
        status = dec._library().qlora_kv_attention(by(cache), by(batch), by(view(q, heads)), by(view(room[32:], heads)), dim ** -0.5, tokens,
                                                   length, (ws.data_ptr() + 255) // 256 * 256, size, torch.cuda.current_stream().cuda_stream)
        assert status == nf4.NF4_OK
        torch.cuda.synchronize()
        assert (room[:32] == 7).all() and (room[32 + tokens:] == 7).all()
        if wrong[0] < 0 < wrong[1]:
            continue                                                # (the third sequence lays claim to the first one's tokens)
        got = room[32:32 + tokens - 2].float()
        assert torch.all((got - want[:tokens - 2].float()).abs() <= 2.0 ** -7 * got.abs() + 2.0 ** -10 * 8)
    nf4.kv_append(c.cache, c.k, c.v, starts, lengths, table, rope=nf4.rope_plan(64), q=c.q)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("counts", [[2, 1, 3], [60, 1, 3]])
def test_lengths_near_their_limit(dim, counts):
    # lengths that pass 2^31 with their new tokens, or hold no table: left out, and the third sequence is served
    c = Case([0, 0, 20], counts, page=16, kv=2, heads=6, dim=dim, seed=22)
    for lengths in ([2 ** 31 - 1, 2 ** 31 - 1, 20], [2 ** 31 - 2, 2 ** 31 - 40, 20], [2 ** 30, -2 ** 31, 20]):
        c.lengths = np.array(lengths)
        before = c.cache.codes.clone()
        check_append(c, with_q=True)
        gone = c.table[:2][c.table[:2] >= 0]
        assert torch.equal(c.cache.codes[gone], before[gone])
        out = check_attention(c, max_new=max(counts), max_length=23)
        assert not out[:sum(counts[:2])].any() and out[sum(counts[:2]):].any(-1).all()


def test_attention_of_appended_tokens_and_other_streams():
    # prompts, then single tokens, on a stream of their own: against float64 attention of the decoded cache
    plan = nf4.rope_plan(128, interleaved=True)
    c = Case([0, 0, 0], [70, 1, 33], page=32, kv=2, heads=8, dim=128, seed=15, fill=False, spare=6)
    c.table = np.array([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for step in range(4):
            q = nf4.kv_append(c.cache, c.k, c.v, *c.meta(), rope=plan, q=c.q)
            c.q = q
            check_attention(c, max_new=int(c.counts.max()), max_length=int((c.lengths + c.counts).max()))
            c.lengths = c.lengths + c.counts
            c.counts = np.ones(3, int)
            c.starts = np.arange(4)
            qkv = torch.randn((3, 12, 128), device="cuda").bfloat16()
            c.q, c.k, c.v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    s.synchronize()


def test_offsets_past_32_bits():
    # a pool of over 4 GiB: pages at its end
    pages = (1 << 32) // (2 * 8 * 256 * 256) + 40
    cache = nf4.KVCache(torch.zeros((pages, 2, 8, 256, 256), dtype=torch.uint8, device="cuda"),
                        torch.ones((pages, 2, 8), device="cuda"))
    c = Case([0, 250], [300, 9], page=256, kv=8, heads=8, dim=256, seed=16)
    c.cache = cache
    c.table = np.array([[pages - 1, pages - 2], [pages - 3, 0]])
    k, v = c.k.clone(), c.v.clone()
    q = nf4.kv_append(cache, k, v, *c.meta())
    assert q is None
    low = nf4.KVCache(cache.codes[pages - 3:].clone(), cache.scales[pages - 3:].clone())
    out = nf4.kv_attention(cache, c.q, *c.meta())
    c.cache, c.table = low, np.array([[2, 1], [0, 0]])
    got = low.decode()[2, 1, :, :256]
    assert torch.all((got.transpose(0, 1) - v[:256].float()).abs() <= v[:256].float().abs() * 2.0 ** -4 + 2.0 ** -15)
    low.codes[0, :, :, :250] = 0
    low.codes = torch.cat([low.codes, cache.codes[:1]])
    low.scales = torch.cat([low.scales, cache.scales[:1]])
    c.table = np.array([[2, 1], [0, 3]])
    assert torch.equal(nf4.kv_attention(low, c.q, *c.meta()), out)
    del cache


def test_graph_replays():
    # append and attention captured once, replayed with other inputs in the same buffers
    plan = nf4.rope_plan(128)
    c = Case([40, 7], [1, 1], page=16, kv=2, heads=4, dim=128, seed=17)
    starts, lengths, table = c.meta()
    k, v, q = c.k.contiguous(), c.v.contiguous(), c.q.contiguous()
    keep = nf4.KVCache(c.cache.codes.clone(), c.cache.scales.clone())

    def step(cache):
        rq = nf4.kv_append(cache, k, v, starts, lengths, table, rope=plan, q=q)
        return nf4.kv_attention(cache, rq, starts, lengths, table, max_new=1, max_length=600)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(nf4.KVCache(keep.codes.clone(), keep.scales.clone()))
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c.cache)
    for i in range(4):
        k.normal_()
        v.normal_()
        q.normal_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step(keep))
        assert torch.equal(c.cache.codes, keep.codes) and torch.equal(c.cache.scales, keep.scales)
        lengths += 1


def test_refused_tensors():
    c = Case([0], [2], kv=2, heads=4)
    st, ln, tb = c.meta()
    for bad in (lambda: nf4.kv_append(c.cache, c.k.float(), c.v, st, ln, tb), lambda: nf4.kv_append(c.cache, c.k, c.v[:1], st, ln, tb),
                lambda: nf4.kv_append(c.cache, c.k, c.v, st.long(), ln, tb), lambda: nf4.kv_append(c.cache, c.k, c.v, st[:1], ln, tb),
                lambda: nf4.kv_append(c.cache, c.k, c.v, st, ln, tb[0]), lambda: nf4.kv_append(c.cache, c.k.cpu(), c.v, st, ln, tb),
                lambda: nf4.kv_attention(c.cache, c.q[..., :64], st, ln, tb), lambda: nf4.kv_attention(c.cache, c.q, st, ln, tb.cpu()),
                lambda: nf4.kv_attention(nf4.KVCache(c.cache.codes, c.cache.scales[:1]), c.q, st, ln, tb)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nf4.NF4Error):
        nf4.kv_attention(c.cache, c.q[:, :3], st, ln, tb)             # 3 heads over 2 key heads
    with pytest.raises(nf4.NF4Error):
        nf4.kv_append(c.cache, c.k[:, :1], c.v, st, ln, tb)
