"""Attention with a window over the paged cache on the GPU against float64.  Bounds as in test_gpu_kv."""
import math

import numpy as np
import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import step_ref as ref
from test_gpu_kv import Case, dev, f64

pytestmark = pytest.mark.gpu


def check(c, window, sinks=0, scale=None, **kw):
    codes, scales = c.host()
    out = nf4.kv_attention(c.cache, c.q, *c.meta(), scale=scale, window=window, sinks=sinks, **kw)
    want, reach = ref.attention(codes, scales, f64(c.q), c.starts, c.lengths, c.table, scale or 1 / math.sqrt(c.dim), window, sinks)
    got = f64(out)
    assert np.all(np.isfinite(got))
    err = np.abs(got - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * reach[..., None]), (err / (reach[..., None] + 1e-30)).max()
    return out


def unseen_pages(c, window, sinks):
    """(sequence, page index) of the pages that no new token sees."""
    got = []
    for b, (n, k) in enumerate(zip(c.lengths, c.counts)):
        for p in range(-(-max(0, n + k) // c.page)):
            keys = np.arange(p * c.page, (p + 1) * c.page)
            if k == 0 or not ((keys < sinks) | (keys > n - window)).any():
                got.append((b, p))
    return got


WINDOWS = [(1, 0), (1, 1), (16, 0), (17, 4), (64, 16), (100, 33), (129, 200), (100000, 5)]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 256])
@pytest.mark.parametrize("kv,heads", [(1, 1), (2, 14), (1, 40)])
def test_single_tokens(dim, page, kv, heads):
    c = Case([0, 1, 14, 15, 16, 31, 32, 127, 128, 300, 777], [1] * 11, page=page, kv=kv, heads=heads, dim=dim, seed=dim + heads)
    for window, sinks in WINDOWS:
        check(c, window, sinks, max_new=1, max_length=778)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,heads", [(2, 2), (1, 5), (2, 32)])
@pytest.mark.parametrize("page", [16, 32])
def test_prompts(dim, kv, heads, page):
    c = Case([0, 100, 0, 45, 3, 260], [1, 33, 130, 0, 17, 64], page=page, kv=kv, heads=heads, dim=dim, seed=dim + heads)
    for window, sinks in WINDOWS:
        a = check(c, window, sinks, max_new=130, max_length=330)
    for kw in (dict(max_new=1, max_length=1), dict(max_new=4000, max_length=100000), {}):
        check(c, 40, 3, **kw)
    # a window as long as the sequences is no window
    b = nf4.kv_attention(c.cache, c.q, *c.meta(), max_new=130, max_length=330)
    assert torch.all((a.float() - b.float()).abs() <= 2.0 ** -7 * a.float().abs() + 2.0 ** -10 * 8)


@pytest.mark.parametrize("dim,page,counts", [(128, 64, [300, 290, 45, 0]), (64, 16, [310, 200, 90, 3]), (64, 32, [500, 333, 270, 1]),
                                             (256, 128, [70, 200, 1, 100])])
def test_many_blocks(dim, page, counts):
    c = Case([150, 10, 400, 33], counts, page=page, kv=2, heads=64, dim=dim, seed=sum(counts))
    for window, sinks in ((70, 4), (256, 0)):
        check(c, window, sinks, max_new=max(counts), max_length=550)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 128])
@pytest.mark.parametrize("counts", [[1, 1, 1], [40, 3, 130]])
@pytest.mark.parametrize("window,sinks", [(50, 4), (64, 0), (1, 17), (200, 40)])
def test_pages_that_nobody_sees_are_not_read(dim, page, counts, window, sinks):
    # given back (entries of -1), then given to others, with codes and scales of NaN
    c = Case([900, 333, 1290], counts, page=page, kv=2, heads=8, dim=dim, seed=dim + page)
    clean = check(c, window, sinks, max_new=max(counts), max_length=1300)
    gone = unseen_pages(c, window, sinks)
    assert len(gone) > 3
    table = c.table.copy()
    for b, p in gone:
        table[b, p] = -1
    full, c.table = c.table, table
    assert torch.equal(check(c, window, sinks, max_new=max(counts), max_length=1300), clean)
    for b, p in gone:
        c.cache.codes[full[b, p]] = 127
        c.cache.scales[full[b, p]] = float("nan")
    c.table = full
    got = nf4.kv_attention(c.cache, c.q, *c.meta(), max_new=max(counts), max_length=1300, window=window, sinks=sinks)
    assert torch.equal(got, clean)


def test_keys_of_nan_outside_the_window():
    # a non-finite token inside a page that is read for others
    c = Case([70, 200], [1, 6], page=64, kv=1, heads=2, dim=128, seed=13)
    clean = check(c, 20, 3)
    c.cache.codes[c.table[0, 0], 0, :, 40] = 127
    c.cache.codes[c.table[1, 0], 0, :, 3] = 127
    c.cache.codes[c.table[1, 2], 0, :, 181 - 128] = 127              # the first new token's window begins there
    out = nf4.kv_attention(c.cache, c.q, *c.meta(), window=20, sinks=3)
    assert torch.equal(out[0], clean[0]) and torch.isnan(out[1]).all() and torch.equal(out[2:], clean[2:])


def test_long_sequences():
    c = Case([40000, 3, 20011], [1, 1, 2], page=64, kv=1, heads=4, dim=128, seed=9)
    for window, sinks in ((5000, 4), (30000, 100), (7, 0)):
        check(c, window, sinks, max_new=2, max_length=40001)
    check(c, 5000, 4)


@pytest.mark.parametrize("counts", [[1, 1], [3, 70]])
def test_positions_near_the_end_of_the_table(counts):
    # sequences that end 2^31 - 256 positions on, over a table that holds them: the answer of the same keys early on
    page, pages, window, sinks = 256, (1 << 31) // 256 - 1, 300, 4
    c = Case([800, 800], counts, page=page, kv=2, heads=8, dim=64, seed=5)
    want = check(c, window, sinks, max_new=max(counts), max_length=1024)
    far = (pages - 4) * page                                         # the last four pages: positions 0 .. 1023 moved by `far`
    table = torch.full((2, pages), -1, dtype=torch.int32, device="cuda")
    table[:, 0] = dev(c.table)[:, 0]
    table[:, pages - 4:pages - 4 + c.table.shape[1]] = dev(c.table)
    for longest in (1024, 2 ** 31 - 1):
        got = nf4.kv_attention(c.cache, c.q, dev(c.starts), dev(c.lengths + far), table, max_new=max(counts), max_length=longest, window=window, sinks=sinks)
        assert torch.all((got.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 2.0 ** -10 * 8)


def test_rows_that_see_nothing():
    c = Case([-1, 4, -3, 10], [1, 1, 5, 1], page=16, kv=2, heads=6, dim=64, seed=14)
    for window, sinks in ((2, 0), (2, 3), (100, 1)):
        out = check(c, window, sinks, max_new=5, max_length=11)
        assert not out[0].any() and not out[2:5].any() and out[1].any() and out[5].any()
    c.table[3, 0] = -1
    assert not check(c, 4, 2, max_new=5, max_length=11)[7].any()
    c.lengths[3] = 16                                                # past the table
    assert not check(c, 4, 2, max_new=5, max_length=17)[7].any()
    c.lengths[3] = -2 ** 31
    assert not check(c, 2 ** 31 - 1, 2 ** 30)[7].any()


def test_the_largest_window_is_none():
    for counts in ([1, 1, 1], [30, 1, 77]):
        c = Case([300, 7, 64], counts, page=16, kv=2, heads=8, dim=128, seed=3)
        check(c, 2 ** 31 - 1, 2 ** 30)
        check(c, 2 ** 31 - 1, 0)
        check(c, 1, 2 ** 30)


def test_refusals():
    c = Case([5], [1], page=16, kv=1, heads=1, dim=64)
    for bad in (dict(window=0), dict(window=-3), dict(window=1 << 31), dict(window=4, sinks=-1), dict(window=4, sinks=(1 << 30) + 1)):
        with pytest.raises(nf4.NF4Error):
            nf4.kv_attention(c.cache, c.q, *c.meta(), **bad)
    with pytest.raises(TypeError):
        nf4.kv_attention(c.cache, c.q, *c.meta(), window=2.5)
