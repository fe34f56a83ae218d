"""A recurrent sequence layer made of the sequence operators, as it is trained and served.

    python examples/sequence_layer.py

One projection gives queries, keys and values; queries and keys are normed per head and turned by position in one pass; linear
attention with a decay per head carries the past.  The demo trains the layer to recall (the value that followed an earlier
key), then reads a prompt and continues it token by token from the kept state, and compares the two.
"""

import os
import sys

import torch
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_evaluation_nonlinear_amd as pn  # noqa: E402


class NormRotary(torch.autograd.Function):
    """qk_norm_rotary with its gradient."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, table, positions):
        ctx.save_for_backward(q, k, q_weight, k_weight, table, positions)
        return pn.qk_norm_rotary(q, k, q_weight, k_weight, table, positions)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, table, positions = ctx.saved_tensors
        grads = pn.qk_norm_rotary_backward(dq.contiguous(), dk.contiguous(), q, k, q_weight, k_weight, table, positions)
        return (*grads, None, None)


class LinearAttention(torch.autograd.Function):
    """linear_attention with its gradient; the state's, where one is carried in or on."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, initial_state):
        ctx.save_for_backward(q, k, v, log_decay, initial_state)
        ctx.set_materialize_grads(False)
        return pn.linear_attention(q, k, v, log_decay, initial_state=initial_state)

    @staticmethod
    @once_differentiable
    def backward(ctx, do, d_final):
        q, k, v, log_decay, initial_state = ctx.saved_tensors
        do = torch.zeros((*q.shape[:3], v.shape[-1]), dtype=q.dtype, device=q.device) if do is None else do.contiguous()
        d_final = None if d_final is None else d_final.contiguous()
        dq, dk, dv, d0 = pn.linear_attention_backward(do, q, k, v, log_decay, initial_state=initial_state, d_final_state=d_final)
        return dq, dk, dv, None, d0


class SequenceLayer(torch.nn.Module):
    """H query heads over HK shared key and value heads of D channels; half of each head turns with position."""

    def __init__(self, width, H=4, HK=2, D=64, positions=4096, dtype=torch.float32, device="cuda"):
        super().__init__()
        self.H, self.HK, self.D = H, HK, D
        self.qkv = torch.nn.Linear(width, (H + 2 * HK) * D, bias=False, dtype=dtype, device=device)
        self.out = torch.nn.Linear(H * D, width, bias=False, dtype=dtype, device=device)
        self.q_weight = torch.nn.Parameter(torch.ones(D, device=device))
        self.k_weight = torch.nn.Parameter(torch.ones(D, device=device))
        # memories of 2^3 .. 2^9 tokens, spread over the heads
        decay = torch.log1p(-torch.exp2(-torch.linspace(3, 9, H, device=device)))
        self.register_buffer("log_decay", decay)
        self.register_buffer("table", pn.rotary_table(positions, pn.rotary_frequencies(D // 2), device=device))

    def heads(self, x):
        """q, k, v as views of the one projection: [B, T, heads, D]."""
        H, HK, D = self.H, self.HK, self.D
        q, k, v = self.qkv(x).split((H * D, HK * D, HK * D), dim=-1)
        return q.unflatten(-1, (H, D)), k.unflatten(-1, (HK, D)), v.unflatten(-1, (HK, D))

    def forward(self, x, state=None, start=None):
        """x [B, T, width] from `state` at position `start` [B] (a fresh sequence: None): (output, state)."""
        q, k, v = self.heads(x)
        B, T = x.shape[:2]
        at = torch.arange(T, device=x.device).expand(B, T) if start is None else start[:, None] + torch.arange(T, device=x.device)
        q, k = NormRotary.apply(q, k, self.q_weight, self.k_weight, self.table, at)
        o, state = LinearAttention.apply(q, k, v, self.log_decay, state)
        return self.out(o.flatten(2)), state

    @torch.no_grad()
    def step(self, x, pool, at, slots=None):
        """One token x [B, width] of each sequence, at position at [B], its state in the pool updated in place."""
        q, k, v = self.heads(x[:, None])
        q, k = pn.qk_norm_rotary(q, k, self.q_weight, self.k_weight, self.table, at[:, None])
        o = pn.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], self.log_decay, pool, slots=slots)
        return self.out(o.flatten(1))


def recall_batch(B, pairs, symbols, generator):
    """Sequences of (key, value) pairs, then a key again: the answer is its value."""
    keys = torch.stack([torch.randperm(symbols, generator=generator)[:pairs] for _ in range(B)])
    values = torch.randint(symbols, 2 * symbols, (B, pairs), generator=generator)
    asked = torch.randint(0, pairs, (B, 1), generator=generator)
    text = torch.cat((torch.stack((keys, values), -1).flatten(1), keys.gather(1, asked)), 1)
    return text.cuda(), values.gather(1, asked)[:, 0].cuda()


class Recall(torch.nn.Module):
    def __init__(self, symbols, width=128, layers=2, **kw):
        super().__init__()
        self.embed = torch.nn.Embedding(2 * symbols, width, device="cuda")
        self.layers = torch.nn.ModuleList(SequenceLayer(width, **kw) for _ in range(layers))
        self.norms = torch.nn.ModuleList(torch.nn.LayerNorm(width, device="cuda") for _ in range(layers + 1))
        self.head = torch.nn.Linear(width, 2 * symbols, device="cuda")

    def forward(self, text):
        x, states = self.embed(text), []
        for layer, norm in zip(self.layers, self.norms):
            y, s = layer(norm(x))
            x = x + y
            states.append(s)
        return self.head(self.norms[-1](x)), states

    @torch.no_grad()
    def step(self, token, pools, at):
        x = self.embed(token)
        for layer, norm, pool in zip(self.layers, self.norms, pools):
            x = x + layer.step(norm(x), pool, at)
        return self.head(self.norms[-1](x))


def train(model, steps, symbols, pairs, B=64, seed=0):
    g = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=3e-3, weight_decay=0.0)
    losses = []
    for _ in range(steps):
        text, answer = recall_batch(B, pairs, symbols, g)
        loss = torch.nn.functional.cross_entropy(model(text)[0][:, -1], answer)
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


def main():
    torch.manual_seed(0)
    symbols, pairs = 16, 8
    model = Recall(symbols)
    losses = train(model, 300, symbols, pairs)
    print(f"recall of {pairs} pairs: loss {losses[0]:.3f} -> {sum(losses[-10:]) / 10:.3f}")
    text, _ = recall_batch(4, pairs, symbols, torch.Generator().manual_seed(1))
    with torch.no_grad():
        whole, _ = model(text)
        _, pools = model(text[:, :9])                     # the prompt; its states are the pools of the steps
        for t in range(9, text.shape[1]):
            one = model.step(text[:, t], pools, torch.full((4,), t, device="cuda"))
            print(f"token {t}: steps and prompt differ by {float((one - whole[:, t]).abs().max()):.1e}")


if __name__ == "__main__":
    main()
