"""examples/sequence_model.py: the sequence operators together, trained and served."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sequence_model
    return sequence_model


def test_training_lowers_the_loss(example):
    losses = example.main(steps=60)
    assert all(torch.isfinite(torch.tensor(losses)))
    assert losses[-1] < 0.7 * losses[0]


def test_tokens_one_by_one_continue_a_prompt(example):
    """Serving a prompt of 20 tokens, or 13 and then 7 single ones, gives the same logits within the activations' rounding."""
    m = example.SequenceModel(vocab=50, dim=64, inner=96, dtype=torch.float32)
    tokens = example.counting(3, 20, 50, 1)
    full = torch.full((3,), 20, dtype=torch.int32, device="cuda")
    a = m.prompt(tokens, full, m.new_states(3))
    states = m.new_states(3)
    # the longest prompt is padded: what lies past a sequence's end does not matter
    m.prompt(tokens, torch.full((3,), 13, dtype=torch.int32, device="cuda"), states)
    for t in range(13, 20):
        b = m.token(tokens[:, t].contiguous(), states)
    assert (a - b).abs().max() <= 1e-4 * a.abs().max()


def test_gradients_against_differences(example):
    """The whole step's gradients along random directions, in f32: central differences of the loss with e = 2^-6 are off by its
    third derivative, e^2 ~ 2e-4 relative, and by f32 rounding of the loss, 2^-22 loss / e ~ 6e-5."""
    make = lambda: example.SequenceModel(vocab=20, dim=32, inner=48, nstate=8, dtype=torch.float32, seed=3)  # noqa: E731
    tokens = example.counting(2, 30, 20, 5)
    m = make()
    m.train_step(tokens, lr=0.0)
    g = torch.Generator(device="cuda").manual_seed(1)
    e = 2.0 ** -6
    for k, grad in m.grads.items():
        v = torch.randn(grad.shape, generator=g, device="cuda")
        v /= v.norm()
        loss = []
        for sign in (1, -1):
            n = make()
            n.w[k] = n.w[k] + sign * e * v
            loss.append(n.train_step(tokens, lr=0.0))
        diff, want = (loss[0] - loss[1]) / (2 * e), float((grad * v).sum())
        assert abs(diff - want) <= 5e-3 * float(grad.norm()) + 2e-4, (k, diff, want)
