"""Sequence-layer operators on the GPU where sizes, strides and values are extreme.

Tolerances are those of test_sequence_gpu.py unless a test derives its own.
"""

import numpy as np
import pytest
import torch

import newton_evaluation_nonlinear_amd as pn
from newton_evaluation_nonlinear_amd import sequence as seq
from oracle import sequence as ref
from test_sequence_gpu import DEV, ROUND, TINY, TYPES, _close, _inputs, _np, _oracle, _rand

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _segments(dtype, B, T, H, HK, DK, DV):
    """Segments of the time axis of a forward call, from the workspace that holds the states between them."""
    code = {"f32": 0, "bf16": 1, "f16": 2}[dtype]
    block = seq._ATTENTION(code, B, T, H, HK, DK, DV, 1.0, *[0] * 29)
    n = pn.lib().pn_linear_attention_workspace_bytes(block, 0)
    return 1 if n <= 256 else 1 + n // (4 * B * H * DK * DV)


# ---------------------------------------------------------------- strides


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("st", [1 << 20, 1 << 27, 1 << 33])
def test_one_token_with_any_token_stride(dtype, st):
    """The stride of a single token is never used: a view of every 2^n-th token of a longer text is as good as its copy."""
    a = _inputs(dtype, 2, 1, 4, 2, 32, 64, True, seed=3)
    far = dict(a)
    for n in ("q", "k", "v", "do"):
        _, _, H, D = a[n].shape
        far[n] = a[n].as_strided((2, 1, H, D), (H * D, st, D, 1))
    names = ("q", "k", "v", "log_decay")
    for x, y in zip(pn.linear_attention(*(far[n] for n in names), initial_state=a["initial_state"]),
                    pn.linear_attention(*(a[n] for n in names), initial_state=a["initial_state"])):
        assert torch.equal(x, y)
    kw = dict(initial_state=a["initial_state"], d_final_state=a["d_final_state"])
    for x, y in zip(pn.linear_attention_backward(*(far[n] for n in ("do",) + names), **kw),
                    pn.linear_attention_backward(*(a[n] for n in ("do",) + names), **kw)):
        assert torch.equal(x, y)
    table = pn.rotary_table(4, pn.rotary_frequencies(32), device=DEV)
    assert torch.equal(pn.rotary(far["q"], table), pn.rotary(a["q"], table))


# ---------------------------------------------------------------- norm gradients


def test_norm_gradients_without_key_heads():
    """k with no heads: the gradient of its weight is a sum over nothing."""
    D = 24
    q, k = torch.randn(2, 5, 4, D, device=DEV), torch.empty(2, 5, 0, D, device=DEV)
    qw, kw = torch.rand(D, device=DEV) + 0.5, torch.ones(D, device=DEV)
    table = pn.rotary_table(8, pn.rotary_frequencies(D), device=DEV)
    want = pn.qk_norm_rotary_backward(q, q[:, :, :1], q, q[:, :, :1], qw, None, table)
    for value in (7.0, float("nan")):                     # over memory that held other values
        used = [torch.full((D,), value, device=DEV) for _ in range(64)]
        del used
        dq, dk, dqw, dkw = pn.qk_norm_rotary_backward(q, k, q, k, qw, kw, table)
        assert dk.shape == k.shape and torch.equal(dq, want[0]) and torch.equal(dqw, want[2])
        assert dkw.shape == kw.shape and torch.equal(dkw, torch.zeros_like(kw))


# ---------------------------------------------------------------- long memories


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("B, H, T, segments", [(64, 8, 32768, 1), (1, 8, 65536, 0)])
def test_long_memories_do_not_drift(dtype, B, H, T, segments):
    """A state carried over tokens that add nothing is e^{g T} of itself, and its gradient likewise.

    Bound: of the decay's power (4 roundings, and the float32 exponent's 2^-24 of it per step of the result's size), and one
    rounding for each factor of about 2 that the state fades by, or each segment; nothing else may grow with T."""
    D = 4
    g = torch.Generator().manual_seed(2)
    ld = -torch.tensor([1.3e-7, 1e-6, 3e-6, 1e-5, 3e-5, 9.3e-5, 3e-4, 1e-3], device=DEV)
    s0, dS = (1.0 + torch.rand(B, H, D, D, generator=g).to(DEV) for _ in range(2))
    n = _segments(dtype, B, T, H, H, D, D)
    assert n == segments if segments else n > 1
    print(f"[long memories] {dtype} B={B} T={T} segments={n}", flush=True)
    zero = torch.zeros(1, 1, 1, D, dtype=TYPES[dtype], device=DEV).expand(B, T, H, D)
    one = torch.ones(1, 1, 1, D, dtype=TYPES[dtype], device=DEV).expand(B, T, H, D)
    S = pn.linear_attention(one, zero, one, ld, initial_state=s0, scale=1.0)[1]
    back = pn.linear_attention_backward(zero, one, zero, one, ld, initial_state=s0, d_final_state=dS, scale=1.0)
    g64 = _np(ld)
    fade = np.exp(g64 * T)[None, :, None, None]
    steps = (1.0 + np.abs(g64) * T / np.log(2.0) + n)[None, :, None, None]
    for got, x, what in ((S, s0, "state"), (back[3], dS, "d initial state")):
        want = _np(x) * fade
        _close(got, want, 6 * EPS * steps * want, what)


# ---------------------------------------------------------------- several segments


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("heads", [(4, 2), (4, 4)])
def test_segments_against_the_oracle(dtype, heads):
    """Sequences that end before, at and after the ends of segments, a decay of its own for every head (none, fast, slow,
    growing), states in and out, shared heads.

    c: dk + dv products, at most 12 sums into a state for every 32 tokens, 64 for the decays and the joins."""
    (H, HK), B, T, DK, DV, scale = heads, 6, 1100, 32, 48, 0.3
    n = _segments(dtype, B, T, H, HK, DK, DV)
    assert n > 2
    seg = 32 * (-(-T // 32) // n + (-(-T // 32) % n > 0))
    lengths = [0, seg, seg + 1, T, 5, 2 * seg - 1]
    print(f"[segments] {dtype} H={H} HK={HK}: {n} of {seg} tokens, lengths {lengths}", flush=True)
    a = _inputs(dtype, B, T, H, HK, DK, DV, True, seed=11)
    a["log_decay"] = torch.tensor([float("-inf"), -5.0, -1e-4, 0.01], device=DEV)
    m = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    kw = dict(initial_state=a["initial_state"], scale=scale, lengths=m)
    o, S = pn.linear_attention(a["q"], a["k"], a["v"], a["log_decay"], **kw)
    c32 = (DK + DV + 12 * T / 32 + 64) * EPS
    c, u, tiny = c32 + (0.0 if dtype == "f32" else 4 * 2.0 ** -16), ROUND[dtype], TINY[dtype]
    top = 65504.0 if dtype == "f16" else np.inf           # with the growing decay some outputs pass binary16's largest number

    def close(got, want, bound, what):
        _close(got.double().clamp(-top, top), np.clip(want, -top, top), bound, what)

    (wo, wS), (Ao, AS) = _oracle(ref.linear_attention, a, ("q", "k", "v", "log_decay", "initial_state"), scale=scale, lengths=lengths)
    close(o, wo, u * np.abs(wo) + c * Ao + tiny, "o")
    _close(S, wS.astype(np.float32).astype(np.float64), c32 * AS, "final state")
    got = pn.linear_attention_backward(a["do"], a["q"], a["k"], a["v"], a["log_decay"], d_final_state=a["d_final_state"], **kw)
    want, mag = _oracle(ref.linear_attention_backward, a, ("do", "q", "k", "v", "log_decay", "initial_state", "d_final_state"),
                        scale=scale, lengths=lengths)
    for name, x, w, A in zip(("dq", "dk", "dv"), got, want, mag):
        close(x, w, u * np.abs(w) + c * A + tiny, name)
    _close(got[3], want[3].astype(np.float32).astype(np.float64), c32 * mag[3], "d initial state")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("DK, DV", [(256, 256), (200, 130), (130, 20), (20, 132), (96, 100), (40, 128), (33, 7)])
def test_segments_of_every_width(dtype, DK, DV):
    """The pass for the segments' states at each number of rows and columns it is built for, read 16 bytes and one channel
    at a time; bounds as in test_segments_against_the_oracle."""
    B, T, H, HK, scale, lengths = 2, 530, 2, 1, 0.3, [530, 333]
    n = _segments(dtype, B, T, H, HK, DK, DV)
    assert n > 1
    print(f"[segments] {dtype} {DK} x {DV}: {n}", flush=True)
    a = _inputs(dtype, B, T, H, HK, DK, DV, True, seed=12)
    kw = dict(initial_state=a["initial_state"], scale=scale, lengths=torch.tensor(lengths, dtype=torch.int32, device=DEV))
    o, S = pn.linear_attention(a["q"], a["k"], a["v"], a["log_decay"], **kw)
    c32 = (DK + DV + 12 * T / 32 + 64) * EPS
    c, u, tiny = c32 + (0.0 if dtype == "f32" else 4 * 2.0 ** -16), ROUND[dtype], TINY[dtype]
    (wo, wS), (Ao, AS) = _oracle(ref.linear_attention, a, ("q", "k", "v", "log_decay", "initial_state"), scale=scale, lengths=lengths)
    _close(o, wo, u * np.abs(wo) + c * Ao + tiny, "o")
    _close(S, wS, c32 * AS, "final state")
    got = pn.linear_attention_backward(a["do"], a["q"], a["k"], a["v"], a["log_decay"], d_final_state=a["d_final_state"], **kw)
    want, mag = _oracle(ref.linear_attention_backward, a, ("do", "q", "k", "v", "log_decay", "initial_state", "d_final_state"),
                        scale=scale, lengths=lengths)
    for name, x, w, A in zip(("dq", "dk", "dv"), got, want, mag):
        _close(x, w, u * np.abs(w) + c * A + tiny, name)
    _close(got[3], want[3], c32 * mag[3], "d initial state")


# ---------------------------------------------------------------- non-finite values


@pytest.mark.parametrize("dtype", list(TYPES))
def test_nan_reaches_at_most_31_tokens_the_other_way(dtype):
    """Of a NaN token: the outputs from it on; of the ones before it at most 31; in the gradients of k and v, which run
    backwards, the tokens after it; other heads and sequences not at all."""
    a = _inputs(dtype, 2, 300, 2, 2, 32, 32, False)
    at, args = 200, ("q", "k", "v", "log_decay")
    clean = pn.linear_attention(*(a[n] for n in args))[0]
    for name in ("k", "v"):
        x = {**a, name: a[name].clone()}
        x[name][1, at, 1] = float("nan")
        o = pn.linear_attention(*(x[n] for n in args))[0]
        assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :, 0], clean[1, :, 0]), name
        assert torch.equal(o[1, :at - 31, 1], clean[1, :at - 31, 1]), name
        assert bool(torch.isnan(o[1, at:, 1]).all()), name
    clean = pn.linear_attention_backward(*(a[n] for n in ("do",) + args))
    for name in ("q", "do"):
        x = {**a, name: a[name].clone()}
        x[name][1, at, 1] = float("nan")
        got = pn.linear_attention_backward(*(x[n] for n in ("do",) + args))
        for y, z in zip(got[1:3], clean[1:3]):            # dk, dv
            assert torch.equal(y[0], z[0]) and torch.equal(y[1, :, 0], z[1, :, 0]), name
            assert torch.equal(y[1, at + 32:, 1], z[1, at + 32:, 1]), name
            assert bool(torch.isnan(y[1, :at + 1, 1]).all()), name


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("DV", [32, 7])
def test_step_keeps_infinities(dtype, DV):
    """lam S + k v of an infinite S is that infinity, for any decay above 0; of the others nothing changes."""
    B, H, DK = 2, 4, 16
    a = _inputs(dtype, B, 1, H, H, DK, DV, True, seed=9)
    a["log_decay"] = torch.tensor([0.0, -1e-5, -0.3, -3.0], device=DEV)
    state = a["initial_state"].clone()
    state[:, :, 3, 2], state[:, :, 5, 4] = float("inf"), float("-inf")
    clean = a["initial_state"].clone()
    pn.linear_attention_step(a["q"][:, 0], a["k"][:, 0], a["v"][:, 0], a["log_decay"], clean)
    pn.linear_attention_step(a["q"][:, 0], a["k"][:, 0], a["v"][:, 0], a["log_decay"], state)
    clean[:, :, 3, 2], clean[:, :, 5, 4] = float("inf"), float("-inf")
    assert torch.equal(state, clean)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T", [1, 70, 1100])
def test_prompts_keep_infinities(dtype, T):
    """An infinite element of the initial state is infinite in the final one, reaches the outputs of its channel as NaN or
    infinity, and nothing else."""
    B, H, DK, DV = 2, 4, 16, 40
    a = _inputs(dtype, B, T, H, H, DK, DV, True, seed=9)
    a["log_decay"] = torch.tensor([0.0, -1e-5, -1e-3, 1e-3], device=DEV)
    args = (a["q"], a["k"], a["v"], a["log_decay"])
    o, S = pn.linear_attention(*args, initial_state=a["initial_state"])
    a["initial_state"][:, :, 3, 2], a["initial_state"][:, :, 5, 34] = float("inf"), float("-inf")
    y, R = pn.linear_attention(*args, initial_state=a["initial_state"])
    S[:, :, 3, 2], S[:, :, 5, 34] = float("inf"), float("-inf")
    assert torch.equal(R, S)
    rest = [c for c in range(DV) if c not in (2, 34)]
    assert torch.equal(y[..., rest], o[..., rest]) and not bool(torch.isfinite(y[..., [2, 34]]).any())


# ---------------------------------------------------------------- launches past 2^32 threads


def test_shared_head_gradients_past_2_32_elements():
    """With a state that holds the current token only and v = do = 1, dk is the sum of scale q over the heads that share it:
    exact in float32, so that every one of 2^32 elements is known to the bit."""
    B, T, H, HK, D = 16, 65536, 64, 32, 128
    q = _rand(torch.Generator().manual_seed(1), (1, 1, H, D), "bf16")
    one = torch.ones(1, 1, 1, 1, dtype=torch.bfloat16, device=DEV)
    ld = torch.full((H,), float("-inf"), device=DEV)
    print("[shared heads] 2^32 elements", flush=True)
    _, dk, dv, _ = pn.linear_attention_backward(one.expand(B, T, H, 1), q.expand(B, T, H, D), q[:, :, :HK].expand(B, T, HK, D),
                                                one.expand(B, T, HK, 1), ld, scale=0.5)
    want = (0.5 * q.float()).view(HK, 2, D).sum(1).bfloat16()
    for b in range(B):
        assert bool((dk[b] == want).all()), b
    assert bool((dv == dv[:1, :1]).all())


def test_rotary_past_2_32_threads():
    T, D = 1 << 27, 33                                    # single channels: 32 lanes a row
    x = _rand(torch.Generator().manual_seed(1), (1, 1, 1, D), "bf16")
    table = pn.rotary_table(8, pn.rotary_frequencies(2), device=DEV)
    at = torch.tensor([3], device=DEV)
    print("[rotary] 2^27 rows of 33 channels", flush=True)
    y = pn.rotary(x.expand(1, T, 1, D), table, at.expand(T))
    want = pn.rotary(x, table, at)
    for t in range(0, T, T // 16):
        assert bool((y[:, t:t + T // 16] == want).all()), t


def test_rotary_table_past_2_32_entries():
    n_pos, n_freq = 1 << 25, 128
    f = pn.rotary_frequencies(2 * n_freq)
    print("[rotary table] 2^32 entries", flush=True)
    t = pn.rotary_table(n_pos, f, device=DEV)
    at = np.array([0, 1, 12345, n_pos // 2, n_pos - 2, n_pos - 1])
    got = _np(t[torch.tensor(at, device=DEV)])
    c, s = ref.angles(at, f)
    assert np.all(np.abs(got[..., 0] - c) <= EPS * np.abs(c) + 2.0 ** -50 * n_pos)
    assert np.all(np.abs(got[..., 1] - s) <= EPS * np.abs(s) + 2.0 ** -50 * n_pos)


def test_norm_gradients_of_many_heads():
    """A weight for each of 70000 heads: more sums than a launch has workgroups along y."""
    H, D, eps = 70000, 2, 1e-5
    g = torch.Generator().manual_seed(8)
    q, dy = _rand(g, (1, 2, H, D), "f32"), _rand(g, (1, 2, H, D), "f32")
    w = 1.0 + 0.3 * _rand(g, (H, D), "f32")
    table = pn.rotary_table(4, pn.rotary_frequencies(D), device=DEV)
    none = q[:, :, :0]
    dq, _, dqw, _ = pn.qk_norm_rotary_backward(dy, none, q, none, w, None, table, eps=eps)
    t = _np(table)[np.arange(2)][None]
    dx, dw, bdx, bdw = ref.norm_rotate_backward(_np(dy), _np(q), _np(w), t[..., 0], t[..., 1], eps)
    _close(dq, dx, EPS * np.abs(dx) + (3 * D + 32) * EPS * bdx, "dq")
    _close(dqw, dw, (2 + D + 16) * EPS * bdw, "dw")


# ---------------------------------------------------------------- refusals


def test_heads_without_channels_are_refused():
    """As the library refuses them, with its error, not with one of the default scale."""
    x, v, g = torch.zeros(1, 2, 1, 0, device=DEV), torch.zeros(1, 2, 1, 4, device=DEV), torch.zeros(1, device=DEV)
    for call in (lambda: pn.linear_attention(x, x, v, g), lambda: pn.linear_attention_backward(v, x, x, v, g),
                 lambda: pn.linear_attention_step(x[:, 0], x[:, 0], v[:, 0], g, torch.zeros(1, 1, 0, 4, device=DEV))):
        with pytest.raises(pn.PnError) as e:
            call()
        assert e.value.code == pn.EUNSUPPORTED
