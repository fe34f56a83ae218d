"""The state-space operators together, in the example's blocks: gradients against differences, a prompt against single
tokens and against two halves, a training step captured beside an eager one."""

import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import state_space_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def test_model_gradients_against_differences():
    torch.manual_seed(0)
    model = ex.Model(6, width=32, layers=2, N=5, W=3)
    text = ex.marked_batch(2, 20, 3, 6, torch.Generator().manual_seed(0))
    up = torch.randn(2, 23, 6, device="cuda")
    with torch.no_grad():
        for p in model.parameters():
            p += 0.05 * torch.randn_like(p)

    def loss():
        return (model(text)[0].double() * up).sum()

    loss().backward()
    for name, t in model.named_parameters():
        d = torch.randn_like(t)
        d /= d.norm()
        h = 2e-2 / (1.0 + float(t.grad.norm()) / 20)
        with torch.no_grad():
            values = []
            for k in (-2, -1, 1, 2):
                t += k * h * d
                values.append(float(loss()))
                t -= k * h * d
        # fourth-order difference: its own error h^4 f^(5) / 30 and the rounding of float32 losses of size 1e2
        diff = (values[0] - 8 * values[1] + 8 * values[2] - values[3]) / (12 * h)
        grad = float((t.grad.double() * d).sum())
        assert abs(diff - grad) <= 1e-2 * (1.0 + float(t.grad.norm())), (name, diff, grad)


def test_state_gradients_against_differences():
    torch.manual_seed(1)
    block = ex.StateSpaceBlock(16, N=8)
    u = torch.randn(2, 9, 16, device="cuda", requires_grad=True)
    past = torch.randn(2, 3, 32, device="cuda", requires_grad=True)
    h0 = torch.randn(2, 32, 8, device="cuda", requires_grad=True)
    up = [torch.randn(2, 9, 16, device="cuda"), torch.randn(2, 3, 32, device="cuda"), torch.randn(2, 32, 8, device="cuda")]

    def loss():
        y, (p, h) = block(u, (past, h0))
        return sum((a.double() * b).sum() for a, b in zip((y, p, h), up))

    loss().backward()
    for t in (u, past, h0):
        d = torch.randn_like(t)
        d /= d.norm()
        h = 1e-2
        with torch.no_grad():
            values = []
            for k in (-2, -1, 1, 2):
                t += k * h * d
                values.append(float(loss()))
                t -= k * h * d
        diff = (values[0] - 8 * values[1] + 8 * values[2] - values[3]) / (12 * h)
        grad = float((t.grad.double() * d).sum())
        assert abs(diff - grad) <= 1e-2 * (1.0 + float(t.grad.norm())), tuple(t.shape)


def test_prompt_single_tokens_and_halves_agree():
    torch.manual_seed(2)
    model = ex.Model(8)
    text = ex.marked_batch(3, 40, 4, 8, torch.Generator().manual_seed(2))
    with torch.no_grad():
        whole, _ = model(text)
        first, states = model(text[:, :17])
        rest, _ = model(text[:, 17:], states)
        assert float((torch.cat((first, rest), 1) - whole).abs().max()) <= 1e-4
        # the pools: rows of their own, the other way round
        slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
        pools = [tuple(torch.zeros(5, *s.shape[1:], dtype=s.dtype, device="cuda").index_copy(0, slots.long(), s) for s in st)
                 for st in states]
        for t in range(17, text.shape[1]):
            one = model.step(text[:, t], pools, slots)
            assert float((one - whole[:, t]).abs().max()) <= 1e-4


def test_a_captured_step_is_the_eager_one():
    torch.manual_seed(3)
    model = ex.Model(8)
    text = ex.marked_batch(4, 12, 2, 8, torch.Generator().manual_seed(3))
    with torch.no_grad():
        _, states = model(text[:, :5])
        held = [tuple(t.clone() for t in st) for st in states]
        token = text[:, 5].clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            model.step(token, [tuple(t.clone() for t in st) for st in states])
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = model.step(token, held)
        for t in range(5, text.shape[1]):
            token.copy_(text[:, t])
            graph.replay()
            want = model.step(text[:, t], states)
            torch.cuda.synchronize()
            assert torch.equal(out, want)
            assert all(torch.equal(a, b) for x, y in zip(held, states) for a, b in zip(x, y))


def test_training_runs():
    torch.manual_seed(0)
    losses = ex.train(ex.Model(5, width=32), 5, 5, T=10, marks=2, B=4)
    assert len(losses) == 5 and all(x == x and x < float("inf") for x in losses)


def test_second_derivatives_are_refused():
    block = ex.StateSpaceBlock(8, N=4)
    u = torch.randn(1, 4, 8, device="cuda", requires_grad=True)
    d, = torch.autograd.grad(block(u)[0].square().sum(), u, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d.sum().backward()
