"""The example decoder: training and serving read the same model."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import small_decoder as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def sequence(n, seed):
    text = torch.randint(0, ex.VOCAB, (n,), generator=torch.Generator().manual_seed(seed)).tolist()
    tokens, targets = torch.tensor(text[:-1], device="cuda"), torch.tensor(text[1:], device="cuda")
    return text, tokens, targets


@pytest.fixture(scope="module")
def trained():
    model = ex.Decoder()
    text, tokens, targets = sequence(97, 1)
    targets[:15] = -100
    return model, text, tokens, targets, ex.train(model, tokens, targets)


def test_adapters_learn(trained):
    losses = trained[4]
    assert all(x == x for x in losses) and losses[-1] < 0.5 * losses[0]


def test_gradient_against_differences():
    # along the gradient's own direction the loss changes by its norm: a step of h changes it by h |d| within the
    # curvature (second order in h) and bf16's rounding of the activations (2^-8 of logits of order 1, averaged)
    model = ex.Decoder(seed=3)
    _, tokens, targets = sequence(80, 4)
    model.table.requires_grad_(True)
    ex.train_loss(model, tokens, targets).backward()
    layer = model.layers[0]["qkv"]
    d = layer.gradients[1]                                     # dB of the first layer: through attention and rope
    unit = d / d.norm()
    base, h = layer.B.float(), 0.5
    losses = []
    for sign in (1, -1):
        layer.B = (base + sign * h * unit).bfloat16()
        losses.append(float(ex.train_loss(model, tokens, targets).detach()))
    slope = (losses[0] - losses[1]) / (2 * h)
    assert abs(slope - float(d.norm())) <= 0.1 * float(d.norm())


def test_cache_serves_what_was_trained(trained):
    # E4M3 keys and values: 2^-4 of a value at most, 2^-5.3 on average, of independent signs, so attention's outputs
    # and with them the logits (of order 1 to 10 after training) move by a few percent each
    model, text, tokens, targets, _ = trained
    want = float(ex.train_loss(model, tokens, targets).detach())
    assert abs(ex.Server(model, 1, 128).score(text, 16) - want) <= 0.1 * max(1.0, want)


def test_batch_answers_as_alone(trained):
    model, text = trained[0], trained[1]
    prompts = [text[:16], text[:40], text[:23]]
    together = ex.Server(model, 3, 64).answer(prompts, 8)
    good = sum(t == w for p, a in zip(prompts, together) for t, w in zip(a, text[len(p):]))
    assert [len(a) for a in together] == [8, 8, 8] and good >= 12       # a learnt text is mostly given back
