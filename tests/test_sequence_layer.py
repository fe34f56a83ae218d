"""The example layer: its gradients against differences, and reading a prompt against single tokens."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import sequence_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_layer_gradients_against_differences():
    torch.manual_seed(0)
    layer = ex.SequenceLayer(24, H=2, HK=1, D=16, positions=64)
    x = torch.randn(2, 37, 24, device="cuda", requires_grad=True)
    s0 = torch.randn(2, 2, 16, 16, device="cuda", requires_grad=True)
    a, b = torch.randn(2, 37, 24, device="cuda"), torch.randn(2, 2, 16, 16, device="cuda")

    def loss():
        y, s = layer(x, s0, torch.tensor([3, 11], device="cuda"))
        return (y.double() * a).sum() + (s.double() * b).sum()

    loss().backward()
    for t in (x, s0, layer.qkv.weight, layer.out.weight, layer.q_weight, layer.k_weight):
        d = torch.randn_like(t)
        d /= d.norm()
        h = 2e-2
        with torch.no_grad():
            values = []
            for k in (-2, -1, 1, 2):
                t += k * h * d
                values.append(float(loss()))
                t -= k * h * d
        # fourth-order difference: its own error h^4 f^(5) / 30 and the rounding of float32 losses of size 1e3
        diff = (values[0] - 8 * values[1] + 8 * values[2] - values[3]) / (12 * h)
        grad = float((t.grad.double() * d).sum())
        assert abs(diff - grad) <= 1e-2 * (1.0 + float(t.grad.norm())), tuple(t.shape)


def test_prompt_and_single_tokens_agree():
    torch.manual_seed(1)
    model = ex.Recall(16)
    text, _ = ex.recall_batch(3, 8, 16, torch.Generator().manual_seed(2))
    with torch.no_grad():
        whole, _ = model(text)
        _, pools = model(text[:, :5])
        for t in range(5, text.shape[1]):
            one = model.step(text[:, t], pools, torch.full((3,), t, device="cuda"))
            assert float((one - whole[:, t]).abs().max()) <= 1e-4


def test_training_lowers_the_loss():
    torch.manual_seed(0)
    model = ex.Recall(8)
    losses = ex.train(model, 60, 8, 4, B=32)
    assert sum(losses[-10:]) < 0.7 * sum(losses[:10])


def test_second_derivatives_are_refused():
    """The gradients are calls of their own, not differentiable ones: asked for theirs, they say so."""
    layer = ex.SequenceLayer(8, H=1, HK=1, D=8, positions=8)
    x = torch.randn(1, 4, 8, device="cuda", requires_grad=True)
    s0 = torch.zeros(1, 1, 8, 8, device="cuda", requires_grad=True)
    y, _ = layer(x, s0)
    d, = torch.autograd.grad(y.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d.sum().backward()
