"""Attention with windows that cut some sequences of a batch, or none of them, against float64.  Bounds as in test_gpu_window."""
import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
from test_gpu_kv import Case
from test_gpu_window import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,kv,heads", [(64, 2, 6), (128, 1, 8), (256, 1, 3)])
def test_one_long_sequence_among_short_ones(dim, kv, heads):
    # windows of one chunk, of several and of more than the sequences' keys; the long one first, inside and last
    for place in (0, 5, 11):
        before = [200 + 7 * i for i in range(12)]
        before[place] = 30000
        c = Case(before, [1] * 12, page=64, kv=kv, heads=heads, dim=dim, seed=dim + place)
        for window, sinks in ((4000, 4), (20000, 0), (40000, 4)):
            a = check(c, window, sinks, max_new=1, max_length=30001)
            assert torch.equal(a, nf4.kv_attention(c.cache, c.q, *c.meta(), max_new=1, max_length=30001, window=window, sinks=sinks))


@pytest.mark.parametrize("counts", [[300, 290, 45, 0], [3, 500, 2, 1]])
def test_prompts_behind_windows_of_any_share(counts):
    # blocks start in the order of their keys where the window is at least half of the longest sequence
    c = Case([150, 10, 400, 33], counts, page=32, kv=4, heads=64, dim=128, seed=sum(counts))
    for window in (60, 274, 275, 276, 400, 549, 550, 551, 5000):
        check(c, window, 0, max_new=max(counts), max_length=550)
