"""State-space blocks made of the state-space operators, as they are trained and served.

    python examples/state_space_layer.py

A block projects its input to x and a gate, convolves x over the last few tokens, derives the scan's steps, b and c from it and
runs the selective scan with the gate; the norm between blocks adds the block's output, normed and scaled, to the residual
stream and prepares the next block's input in the same pass.  The demo trains two blocks to repeat the symbols of a text that
are marked, then reads a prompt and continues it token by token from the kept states, and compares the two.
"""

import math
import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_evaluation_nonlinear_amd as pn  # noqa: E402


def _dense(g, like):
    """A gradient that may be missing or strided by 0, as the calls take it."""
    return torch.zeros_like(like) if g is None else g.contiguous()


class ShortConv(torch.autograd.Function):
    """short_conv with its gradient: (y, the last tokens)."""

    @staticmethod
    def forward(ctx, x, weight, bias, initial_state):
        ctx.save_for_backward(x, weight, bias, initial_state)
        ctx.set_materialize_grads(False)
        return pn.short_conv(x, weight, bias=bias, initial_state=initial_state)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, d_final):
        x, weight, bias, initial_state = ctx.saved_tensors
        return pn.short_conv_backward(_dense(dy, x), x, weight, bias=bias, initial_state=initial_state,
                                      d_final_state=None if d_final is None else d_final.contiguous())


class Scan(torch.autograd.Function):
    """ssm_scan with its gradient: (y, the state after the last token)."""

    @staticmethod
    def forward(ctx, x, dt, A, b, c, skip, gate, dt_bias, initial_state):
        ctx.save_for_backward(x, dt, A, b, c, skip, gate, dt_bias, initial_state)
        ctx.set_materialize_grads(False)
        return pn.ssm_scan(x, dt, A, b, c, skip=skip, gate=gate, dt_bias=dt_bias, initial_state=initial_state)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, d_final):
        x, dt, A, b, c, skip, gate, dt_bias, initial_state = ctx.saved_tensors
        return pn.ssm_scan_backward(_dense(dy, x), x, dt, A, b, c, skip=skip, gate=gate, dt_bias=dt_bias, initial_state=initial_state,
                                    d_final_state=None if d_final is None else d_final.contiguous())


class BlockNorm(torch.autograd.Function):
    """block_norm with its gradient: (the next block's input, the residual stream)."""

    @staticmethod
    def forward(ctx, x, residual, weight, post_weight, scale):
        ctx.save_for_backward(x, residual, weight, post_weight, scale)
        ctx.set_materialize_grads(False)
        return pn.block_norm(x, weight, residual=residual, post_weight=post_weight, scale=scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, ds):
        x, residual, weight, post_weight, scale = ctx.saved_tensors
        dx, dw, dr, _, dpw, dsc = pn.block_norm_backward(_dense(dy, x), None if ds is None else ds.contiguous(), x, weight,
                                                         residual=residual, post_weight=post_weight, scale=scale)
        return dx, dr, dw, dpw, dsc


class StateSpaceBlock(torch.nn.Module):
    """width -> channels (twice the width) with N states each; steps from a projection of low rank."""

    def __init__(self, width, N=16, W=4, dtype=torch.float32, device="cuda"):
        super().__init__()
        D = self.D = 2 * width
        self.N, self.rank = N, max(1, width // 16)
        linear = lambda i, o: torch.nn.Linear(i, o, bias=False, dtype=dtype, device=device)  # noqa: E731
        self.enter, self.leave = linear(width, 2 * D), linear(D, width)
        self.derive, self.steps = linear(D, self.rank + 2 * N), linear(self.rank, D)
        self.conv_weight = torch.nn.Parameter(torch.randn(D, W, device=device) * W ** -0.5)
        self.conv_bias = torch.nn.Parameter(torch.zeros(D, device=device))
        # rates 1 .. N, kept negative through their logarithm; steps of 0.001 to 0.1
        self.log_rate = torch.nn.Parameter(torch.log(torch.arange(1, N + 1, device=device).float()).repeat(D, 1))
        self.skip = torch.nn.Parameter(torch.ones(D, device=device))
        step = torch.exp(torch.rand(D, device=device) * math.log(100.0) + math.log(0.001))
        self.dt_bias = torch.nn.Parameter(step + torch.log(-torch.expm1(-step)))

    def derived(self, x):
        """dt, b and c of the convolved x."""
        r, b, c = self.derive(x).split((self.rank, self.N, self.N), dim=-1)
        return self.steps(r), b.unsqueeze(-2), c.unsqueeze(-2)

    def forward(self, u, state=None):
        """u [B, T, width] from `state` (conv, scan), a fresh sequence: None.  Returns (output, state)."""
        x, gate = self.enter(u).split(self.D, dim=-1)
        past, h = (None, None) if state is None else state
        x, past = ShortConv.apply(x, self.conv_weight, self.conv_bias, past)
        dt, b, c = self.derived(x)
        y, h = Scan.apply(x, dt, -torch.exp(self.log_rate), b, c, self.skip, gate, self.dt_bias, h)
        return self.leave(y), (past, h)

    @torch.no_grad()
    def step(self, u, pool, slots=None):
        """One token u [B, width] of each sequence; the pools (conv, scan) are updated in place."""
        x, gate = self.enter(u).split(self.D, dim=-1)
        x = pn.short_conv_step(x, self.conv_weight, pool[0], bias=self.conv_bias, slots=slots)
        dt, b, c = self.derived(x)
        y = pn.ssm_step(x, dt, -torch.exp(self.log_rate), b, c, pool[1], skip=self.skip, gate=gate, dt_bias=self.dt_bias, slots=slots)
        return self.leave(y)


class Model(torch.nn.Module):
    def __init__(self, symbols, width=64, layers=2, device="cuda", **kw):
        super().__init__()
        ones = lambda: torch.nn.Parameter(torch.ones(width, device=device))  # noqa: E731
        self.embed = torch.nn.Embedding(symbols, width, device=device)
        self.blocks = torch.nn.ModuleList(StateSpaceBlock(width, device=device, **kw) for _ in range(layers))
        self.weights = torch.nn.ParameterList(ones() for _ in range(layers + 1))       # of the norm before a block, and the last
        self.post = torch.nn.ParameterList(ones() for _ in range(layers))              # of the norm after it
        self.scales = torch.nn.ParameterList(ones() for _ in range(layers))
        self.head = torch.nn.Linear(width, symbols, bias=False, device=device)

    def forward(self, text, states=None):
        x, s = BlockNorm.apply(self.embed(text), None, self.weights[0], None, None)
        left = []
        for i, block in enumerate(self.blocks):
            y, state = block(x, None if states is None else states[i])
            left.append(state)
            x, s = BlockNorm.apply(y, s, self.weights[i + 1], self.post[i], self.scales[i])
        return self.head(x), left

    @torch.no_grad()
    def step(self, token, pools, slots=None):
        x, s = pn.block_norm(self.embed(token), self.weights[0])
        for i, (block, pool) in enumerate(zip(self.blocks, pools)):
            x, s = pn.block_norm(block.step(x, pool, slots), self.weights[i + 1], residual=s, post_weight=self.post[i],
                                 scale=self.scales[i])
        return self.head(x)


def marked_batch(B, T, marks, symbols, generator):
    """Texts in which `marks` places hold a symbol to remember, the others filler (0), then the marks again in their order."""
    text = torch.zeros(B, T, dtype=torch.long)
    keep = torch.randint(1, symbols, (B, marks), generator=generator)
    for b in range(B):
        text[b, torch.randperm(T, generator=generator)[:marks].sort().values] = keep[b]
    return torch.cat((text, keep), 1).cuda()


def train(model, steps, symbols, T=24, marks=3, B=32, seed=0):
    g = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        text = marked_batch(B, T, marks, symbols, g)
        out, _ = model(text[:, :-1])
        loss = torch.nn.functional.cross_entropy(out[:, T - 1:].flatten(0, 1), text[:, T:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def main():
    torch.manual_seed(0)
    symbols = 8
    model = Model(symbols)
    losses = train(model, 300, symbols)
    print(f"marked symbols: loss {losses[0]:.3f} -> {sum(losses[-10:]) / 10:.3f}")
    text = marked_batch(4, 24, 3, symbols, torch.Generator().manual_seed(1))
    with torch.no_grad():
        whole, _ = model(text)
        _, pools = model(text[:, :20])                    # the prompt; its states are the pools of the steps
        for t in range(20, text.shape[1]):
            one = model.step(text[:, t], pools)
            print(f"token {t}: steps and prompt differ by {float((one - whole[:, t]).abs().max()):.1e}")


if __name__ == "__main__":
    main()
