"""The example decoder's training loop with and without clipping."""
import pytest
import torch

from test_gpu_example import ex, sequence

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_norm", [None, 0.5])
def test_training_with_and_without_clipping(max_norm):
    _, tokens, targets = sequence(40, 2)
    lines, quiet, told = [], ex.Decoder(seed=5), ex.Decoder(seed=5)
    a = ex.train(quiet, tokens, targets, steps=2, max_norm=max_norm)
    b = ex.train(told, tokens, targets, steps=2, max_norm=max_norm, say=lines.append)
    assert len(a) == 2 and a == b and all(x == x for x in a)
    assert [line.startswith("step") for line in lines] == [True, True] and all(("gradients" in line) == (max_norm is not None) for line in lines)
    assert not torch.equal(quiet.layers[0]["qkv"].B, ex.Decoder(seed=5).layers[0]["qkv"].B)
