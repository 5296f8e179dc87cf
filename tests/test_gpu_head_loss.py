"""The vocabulary head's loss and gradients on the GPU against float64.

Bounds.  A logit's fp32 sum of exact products is within 2 sqrt(K) 2^-24 sum|x w| of the exact one
(rounding errors of K additions; the square root for their signs), and so are lse and loss,
with 2^-21 (|lse| + 1) for the base-2 logarithms.  Gradients: each entry of G is rounded to
bf16, at most 2^-8 of it, and so are the outputs: 2^-8 |dX| + 2^-8 |G| |W| + the logits' error."""
import math

import pytest
import torch

import bit_nf4_quantized_09_amd as nf4
import decoder_abi as dec
import decoder_ref as ref

pytestmark = pytest.mark.gpu


def inputs(M, V, K, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn((M, K), generator=g, device="cuda").bfloat16()
    W = (torch.randn((V, K), generator=g, device="cuda") * (std / math.sqrt(K))).bfloat16()
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    dl = torch.randn(M, generator=g, device="cuda") / M
    return X, W, t, dl


def check(X, W, t, dl, need_dw=True, ignore=-100):
    loss, dX, dW = nf4.head_loss(X, W, t, dloss=dl, need_dw=need_dw, ignore_index=ignore)
    only = nf4.head_loss(X, W, t, ignore_index=ignore)
    wl, wx, ww, G, z = ref.head_loss(X, W, t, dl, ignore)
    K = X.shape[1]
    dz = 2 * math.sqrt(K) * 2.0 ** -24 * (X.double().abs() @ W.double().abs().t()).amax(1)
    tol = 2 * dz + 2.0 ** -21 * (z.abs().amax(1) + 1)
    assert torch.all((loss.double() - wl).abs() <= tol)
    assert only[1] is None and only[2] is None and torch.all((only[0].double() - wl).abs() <= tol)
    slack = 2.0 ** -8 + 2 * float(tol.max())
    ex = (dX.double() - wx).abs() - (2.0 ** -8 * wx.abs() + slack * (G @ W.double().abs()))
    assert torch.all(ex <= 1e-30), float(ex.max())
    if need_dw:
        ew = (dW.double() - ww).abs() - (2.0 ** -8 * ww.abs() + slack * (G.t() @ X.double().abs()))
        assert torch.all(ew <= 1e-30), float(ew.max())
    alone = nf4.head_loss(X, W, t, dloss=dl, ignore_index=ignore)
    ex = (alone[1].double() - wx).abs() - (2.0 ** -8 * wx.abs() + slack * (G @ W.double().abs()))
    assert torch.all(ex <= 1e-30), float(ex.max())
    assert torch.all((alone[0].double() - wl).abs() <= tol)
    return loss, dX, dW


@pytest.mark.parametrize("M,V,K", [(1, 1, 64), (1, 1000, 128), (7, 33, 64), (64, 257, 192), (65, 1023, 512), (255, 300, 320),
                                   (257, 513, 64), (130, 5001, 1024), (700, 2000, 576)])
def test_values(M, V, K):
    check(*inputs(M, V, K, seed=M + V))


@pytest.mark.parametrize("M,V,K", [(2, 1211, 704), (32, 129, 64), (33, 4097, 128), (63, 2000, 1088), (64, 50001, 64), (66, 128, 2048),
                                   (128, 1322, 6272), (129, 640, 192), (281, 8191, 256), (513, 1025, 4160), (992, 1524, 576)])
def test_few_tokens_and_small_grids(M, V, K):
    check(*inputs(M, V, K, seed=M + V + K))


@pytest.mark.parametrize("K", [64, 6144])
def test_gradient_past_what_is_kept(K):
    # more than 1 GB of weights: dW from the logits a second time
    check(*inputs(4096, 131200, K, seed=15))


def test_long_contractions():
    check(*inputs(1024, 32000, 6144, seed=17))


@pytest.mark.parametrize("M", [9, 50])
def test_few_tokens_and_pieces_of_the_vocabulary(M):
    check(*inputs(M, 140001, 64, seed=M))


def test_growing_logits_in_pieces():
    # the reference moves within and between pieces whose weights are kept for dW
    X, W, t, dl = inputs(2048, 70000, 64, seed=16)
    X[:, 0] = 1.0
    W[:, 0] = torch.arange(70000, device="cuda").float() / 64
    t[:1024] = 69990
    check(X, W, t, dl)
    W[:, 0] = -W[:, 0].float()
    check(X, W, t, dl)


def test_pieces_of_the_vocabulary():
    # 4096 tokens and 20000 entries: several pieces, a ragged last one
    check(*inputs(4096, 20001, 128, seed=5))


def test_sharp_logits():
    X, W, t, dl = inputs(300, 2000, 256, seed=6, std=40.0)          # logits of some 40: few entries count
    t[::2] = (X.float() @ W.float().t()).argmax(1)[::2]             # half of the targets win
    check(X, W, t, dl)


def test_offset_logits():
    # all logits near +-300: nothing may overflow
    for sign in (1, -1):
        X, W, t, dl = inputs(70, 900, 256, seed=7)
        X[:, 0], W[:, 0] = 300.0 * sign, 1.0
        check(X, W, t, dl)


def test_growing_logits():
    # each later part of the vocabulary dominates all before it by far more than bf16's or fp32's range of exponents
    X, W, t, dl = inputs(520, 40000, 64, seed=8)
    X[:, 0] = 1.0
    W[:, 0] = torch.arange(40000, device="cuda").float() / 16
    t[:260] = 39990
    check(X, W, t, dl, need_dw=False)
    W[:, 0] = -W[:, 0].float()
    check(X, W, t, dl, need_dw=False)


def test_ignored_targets():
    X, W, t, dl = inputs(150, 700, 128, seed=9)
    t[0], t[1], t[2], t[3] = -100, -1, 700, 2 ** 62
    t[10:20] = 5
    loss, dX, dW = check(X, W, t, dl, ignore=5)
    dead = [0, 1, 2, 3] + list(range(10, 20))
    assert not loss[dead].any() and not dX[dead].any()
    t[:] = -100
    loss, dX, dW = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    assert not loss.any() and not dX.any() and not dW.any()
    loss, dX, dW = nf4.head_loss(X, W, t, dloss=dl)
    assert not loss.any() and not dX.any()


@pytest.mark.parametrize("M,V,K", [(3, 500, 64), (33, 2000, 128), (80, 600, 128), (700, 2000, 576), (2048, 40000, 128),
                                   (1024, 32000, 6144), (4096, 131200, 64)])
def test_ignored_rows_hold_anything(M, V, K):
    # what ignored rows of X and dloss hold changes nothing: not even a bit of the others, nor of dW
    X, W, t, dl = inputs(M, V, K, seed=M)
    t[1], t[M - 1] = -100, V
    want = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    only = nf4.head_loss(X, W, t)[0]
    X[1], X[M - 1, 5], dl[1], dl[M - 1] = math.nan, math.inf, math.nan, math.inf
    got = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    assert torch.equal(nf4.head_loss(X, W, t)[0], only)
    assert not got[0][[1, M - 1]].any() and not got[1][[1, M - 1]].any()
    # a row of W that is not finite reaches every row of dX that counts, and no other
    W[V // 2] = math.nan
    for need_dw in (True, False):
        dX = nf4.head_loss(X, W, t, dloss=dl, need_dw=need_dw)[1]
        dead = torch.zeros(M, dtype=torch.bool, device="cuda")
        dead[[1, M - 1]] = True
        assert not dX[dead].any() and torch.isnan(dX[~dead]).all()


def test_non_finite_rows_stay_alone():
    X, W, t, dl = inputs(80, 600, 128, seed=10)
    good = nf4.head_loss(X, W, t, dloss=dl)
    X[3, 5], X[77, 0] = float("nan"), float("inf")
    loss, dX, _ = nf4.head_loss(X, W, t, dloss=dl)
    keep = torch.ones(80, dtype=torch.bool, device="cuda")
    keep[[3, 77]] = False
    assert torch.equal(loss[keep], good[0][keep]) and torch.equal(dX[keep], good[1][keep])
    assert not torch.isfinite(loss[[3, 77]]).any() and not torch.isfinite(dX[[3, 77]]).all(1).any()
    dl2 = dl.clone()
    dl2[9] = float("nan")
    X, W, t, _ = inputs(80, 600, 128, seed=10)
    _, dX, _ = nf4.head_loss(X, W, t, dloss=dl2)
    keep = torch.arange(80, device="cuda") != 9
    assert torch.equal(dX[keep], good[1][keep]) and torch.isnan(dX[9]).all()


@pytest.mark.parametrize("M,V,K", [(3, 500, 64), (80, 600, 128), (700, 2000, 576), (2048, 40000, 128)])
@pytest.mark.parametrize("row", [1, 2])
@pytest.mark.parametrize("sign", [1, -1])
def test_infinite_target_logits(M, V, K, row, sign):
    # a product of 3e38 and 3e38 overflows fp32; every other logit of that row is zero (row 1) or an ordinary one (row 2).
    # With and without gradients the row's loss is the same, and the other rows' are what they were
    X, W, t, dl = inputs(M, V, K, seed=M)
    W[:, 0] = 0
    X[1] = 0
    t[t == t[row]] = (t[row] + 1) % V
    t[row] = (t[row] - 1) % V
    W[t[row], 0] = sign * 3e38
    X[:, 0] = 0
    good = nf4.head_loss(X, W, t, dloss=dl)
    X[row, 0] = 3e38
    alone = nf4.head_loss(X, W, t)[0]
    loss, dX, dW = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    keep = torch.arange(M, device="cuda") != row
    for x in (alone, loss):
        assert torch.isnan(x[row]) if sign > 0 else x[row] == math.inf
        assert torch.all((x[keep] - good[0][keep]).abs() <= 2.0 ** -20 * (good[0][keep].abs() + 1))
    assert torch.equal(dX[keep], good[1][keep])
    if sign > 0:
        assert torch.isnan(dX[row]).all()
        return
    # p of the target is 0: dX = dloss (sum_v p_v W_v - W_y), bounded as in check()
    z = X.double() @ W.double().t()
    z[row, t[row]] = -math.inf
    p = z[row].softmax(0)
    want = dl[row].double() * (p @ W.double() - W[t[row]].double())
    slack = 2.0 ** -8 * want.abs() + 2.0 ** -7 * dl[row].double().abs() * (p @ W.double().abs() + W[t[row]].double().abs())
    assert torch.all((dX[row].double() - want).abs()[1:] <= slack[1:])
    assert torch.isfinite(dW[:, 1:]).all()


def test_equal_factors_lose_nothing():
    # a mean's factor 1/count is no power of two: it must not round every row alike
    X, W, t, _ = inputs(384, 3000, 512, seed=11)
    dl = torch.full((384,), 1 / 367.0, device="cuda")
    _, dX, dW = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    _, wx, ww, _, _ = ref.head_loss(X, W, t, dl)
    # roundings of 2^-9 on average of independent sign, in G and in the output
    for got, want in ((dX, wx), (dW, ww), (nf4.head_loss(X, W, t, dloss=dl)[1], wx)):
        assert float((got.double() - want).norm() / want.norm()) <= 2.5e-3


@pytest.mark.parametrize("M,V,K", [(33, 4000, 512), (64, 20000, 256), (60, 30000, 4096), (384, 3000, 512), (700, 5000, 576),
                                   (2048, 70000, 64), (1024, 32000, 6144)])
@pytest.mark.parametrize("jump", [False, True])
def test_dw_of_rows_without_targets(M, V, K, jump):
    # few tokens, 64-, 256- and 512-row tiles, one piece and several; with `jump` the second half of the vocabulary passes
    # the targets' logits by 60, each tile takes a reference of its own, and they are brought together afterwards
    X, W, t, dl = inputs(M, V, K, seed=3)
    t %= V // 2
    if jump:
        X[:, 0], W[:, 0], W[V // 2:, 0] = 1.0, 0.0, 60.0
    dW = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)[2][V // 2:, 1:].double()
    want = ref.head_loss(X, W, t, dl)[2][V // 2:, 1:]
    assert float((dW - want).norm() / want.norm()) <= ref.DW_NORM


def test_repeats_and_streams():
    X, W, t, dl = inputs(333, 4000, 256, seed=12)
    a = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    s.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_graph_replays():
    X, W, t, dl = inputs(100, 3000, 128, seed=13)
    run = lambda: nf4.head_loss(X, W, t, dloss=dl, need_dw=True)  # noqa: E731
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for i in range(4):
        X.normal_()
        t.random_(0, 3000)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, run()):
            assert torch.equal(x, y)


@pytest.mark.parametrize("M,V,K", [(3, 500, 64), (50, 3000, 128), (300, 5001, 576), (2048, 40000, 64), (4096, 131200, 64)])
def test_each_output_alone(M, V, K):
    # through the C entry any of the outputs may be left out: the others are the same bits
    X, W, t, dl = inputs(M, V, K, seed=19)
    loss, dX, dW = nf4.head_loss(X, W, t, dloss=dl, need_dw=True)
    for with_loss, with_dx, with_dw in ((1, 1, 0), (0, 1, 0), (1, 0, 1), (0, 0, 1), (0, 1, 1)):
        size = dec._library().qlora_head_loss_workspace_bytes(M, K, V, with_dx, with_dw)
        ws = torch.empty(size + 256, dtype=torch.uint8, device="cuda")
        got = [torch.full_like(x, 7.0) if on else None for x, on in ((loss, with_loss), (dX, with_dx), (dW, with_dw))]
        at = [None if x is None else x.data_ptr() for x in got]
        status = dec._library().qlora_head_loss(X.data_ptr(), M, K, W.data_ptr(), V, t.data_ptr(), -100, dl.data_ptr(), *at,
                                                (ws.data_ptr() + 255) // 256 * 256, size, torch.cuda.current_stream().cuda_stream)
        assert status == nf4.NF4_OK
        for x, want in zip(got, (loss, dX, dW)):
            assert x is None or torch.equal(x, want)


def test_nothing():
    X, W, t, dl = inputs(4, 100, 64)
    loss, dX, dW = nf4.head_loss(X[:0], W, t[:0], dloss=dl[:0], need_dw=True)
    assert loss.shape == (0,) and dX.shape == (0, 64) and not dW.any()


def test_refused_tensors():
    X, W, t, dl = inputs(4, 100, 64)
    for bad in (lambda: nf4.head_loss(X.float(), W, t), lambda: nf4.head_loss(X, W[:, :32], t), lambda: nf4.head_loss(X, W, t.int()),
                lambda: nf4.head_loss(X, W, t[:2]), lambda: nf4.head_loss(X, W, t, dloss=dl[:2]), lambda: nf4.head_loss(X, W, t, need_dw=True),
                lambda: nf4.head_loss(X, W, t, dloss=dl.double()), lambda: nf4.head_loss(X.t(), W.t(), t), lambda: nf4.head_loss(X, W.cpu(), t)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nf4.NF4Error):
        nf4.head_loss(X[:, :40].contiguous(), W[:, :40].contiguous(), t)
