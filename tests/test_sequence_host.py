"""Sequence-layer operators without a GPU: the float64 oracle against differences and independent forms, frequency
scalings, and the C entries' refusals (placeholder addresses; nothing is dereferenced)."""

import math

import numpy as np
import pytest
import torch

import newton_evaluation_nonlinear_amd as pn
from newton_evaluation_nonlinear_amd import sequence as seq
from oracle import sequence as ref


@pytest.fixture(autouse=True)
def _no_error_left():
    yield
    pn.lib().pn_rotary(_rotary_block(B=0))               # a call that succeeds clears the thread's message


def _rng(seed=0):
    return np.random.default_rng(seed)


# ---------------------------------------------------------------- oracle pins


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    g = _rng(1)
    x = g.standard_normal((2, 3, 4, 10))
    pos = g.integers(0, 1000, (2, 3))
    f = [1.0, 0.3, 0.01]
    c, s = ref.angles(pos, f)
    y = ref.rotate(x, c, s, interleaved)
    ia, ib = (np.arange(0, 6, 2), np.arange(1, 6, 2)) if interleaved else (np.arange(3), np.arange(3, 6))
    z = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * pos[..., None] * np.array(f))[:, :, None]
    assert np.allclose(y[..., ia], z.real, atol=1e-12) and np.allclose(y[..., ib], z.imag, atol=1e-12)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(ref.rotate(y, c, -s, interleaved), x, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_norm_rotation_gradient_against_differences(interleaved):
    g = _rng(2)
    x, dy, w = g.standard_normal((1, 2, 2, 6)), g.standard_normal((1, 2, 2, 6)), 1 + 0.3 * g.standard_normal((2, 6))
    c, s = ref.angles(np.array([[3, 7]]), [1.0, 0.2])
    dx, dw, _, _ = ref.norm_rotate_backward(dy, x, w, c, s, 1e-3, interleaved)

    def loss(x, w):
        return float(np.sum(dy * ref.rotate(ref.norm(x, w, 1e-3)[0], c, s, interleaved)))

    h = 1e-6
    for a, da in ((x, dx), (w, dw)):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += h
            dn[i] -= h
            d = (loss(up, w) - loss(dn, w) if a is x else loss(x, up) - loss(x, dn)) / (2 * h)
            assert abs(d - da[i]) < 1e-7 * max(1.0, abs(d)) + 1e-7


def test_linear_attention_is_the_masked_product():
    g = _rng(3)
    B, T, H, HK, DK, DV = 2, 9, 4, 2, 3, 5
    q, k, v = g.standard_normal((B, T, H, DK)), g.standard_normal((B, T, HK, DK)), g.standard_normal((B, T, HK, DV))
    ld = np.log(np.array([0.5, 0.9, 0.99, 1.0]))
    S0 = g.standard_normal((B, H, DK, DV))
    n = [9, 4]
    o, S = ref.linear_attention(q, k, v, ld, S0, 0.3, n)
    for b in range(B):
        for h in range(H):
            lam = np.exp(ld[h])
            i = np.arange(n[b])
            M = np.tril(lam ** (i[:, None] - i))
            want = 0.3 * ((q[b, :n[b], h] @ k[b, :n[b], h // 2].T * M) @ v[b, :n[b], h // 2] +
                          lam ** (i[:, None] + 1) * (q[b, :n[b], h] @ S0[b, h]))
            assert np.allclose(o[b, :n[b], h], want, atol=1e-12)
            last = lam ** n[b] * S0[b, h] + sum(lam ** (n[b] - 1 - j) * np.outer(k[b, j, h // 2], v[b, j, h // 2]) for j in i)
            assert np.allclose(S[b, h], last, atol=1e-12)
    assert not o[1, 4:].any()


def test_linear_attention_gradient_against_differences():
    g = _rng(4)
    B, T, H, HK, DK, DV = 2, 5, 2, 1, 2, 3
    a = dict(q=g.standard_normal((B, T, H, DK)), k=g.standard_normal((B, T, HK, DK)), v=g.standard_normal((B, T, HK, DV)),
             S0=g.standard_normal((B, H, DK, DV)))
    ld, n, do, dS = np.log([0.6, 0.95]), [5, 3], g.standard_normal((B, T, H, DV)), g.standard_normal((B, H, DK, DV))
    grads = dict(zip(("q", "k", "v", "S0"), ref.linear_attention_backward(do, a["q"], a["k"], a["v"], ld, a["S0"], dS, 0.7, n)))

    def loss(a):
        o, S = ref.linear_attention(a["q"], a["k"], a["v"], ld, a["S0"], 0.7, n)
        return float(np.sum(o * do) + np.sum(S * dS))

    h = 1e-6
    for name in a:
        for i in np.ndindex(a[name].shape):
            up, dn = {**a, name: a[name].copy()}, {**a, name: a[name].copy()}
            up[name][i] += h
            dn[name][i] -= h
            d = (loss(up) - loss(dn)) / (2 * h)
            assert abs(d - grads[name][i]) < 1e-7 * max(1.0, abs(d)) + 1e-7, (name, i)


# ---------------------------------------------------------------- frequencies


def test_frequency_scalings():
    R, s, L = 64, 4.0, 4096
    f = pn.rotary_frequencies(R)
    assert f[0] == 1.0 and len(f) == 32 and math.isclose(f[16], 10000.0 ** -0.5)
    assert np.allclose(pn.rotary_frequencies(R, scaling="linear", factor=s), np.array(f) / s)
    b = pn.rotary_frequencies(R, scaling="base", factor=s)
    assert b[0] == 1.0 and math.isclose(b[-1], f[-1] / s)
    p = pn.rotary_frequencies(R, scaling="by_parts", factor=s, original_positions=L, low=1.0, high=32.0)
    for x, y in zip(f, p):
        turns = L * x / (2 * math.pi)
        if turns >= 32:
            assert y == x
        elif turns <= 1:
            assert math.isclose(y, x / s)
        else:
            assert x / s < y < x
    for kw in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=8, scaling="other"), dict(rotary_dim=8, base=0.0),
               dict(rotary_dim=8, scaling="by_parts"), dict(rotary_dim=2, scaling="base"), dict(rotary_dim=258),
               dict(rotary_dim=8, scaling="by_parts", original_positions=10, low=2, high=2)):
        with pytest.raises(ValueError):
            pn.rotary_frequencies(**kw)


# ---------------------------------------------------------------- refusals of the C entries

GIB = 1 << 30
TOK = lambda i, sb=64, st=32, sh=8: (i * GIB, sb, st, sh)  # noqa: E731


def _rotary_block(dtype=0, B=2, T=2, D=8, R=4, inter=0, inverse=0, hq=4, hk=4, q=TOK(4), k=TOK(5), qo=6 * GIB, ko=7 * GIB,
                  table=8 * GIB, n_pos=16, pos=0, pos64=0, psb=0, pst=0, off=0, eps=1e-6, qw=0, kw=0, qsh=0, ksh=0,
                  dq=TOK(9), dk=TOK(10), dqw=0, dkw=0, ws=0, wsn=0):
    return seq._ROTARY(dtype, B, T, D, R, inter, inverse, hq, hk, *q, *k, qo, ko, table, n_pos, pos, pos64, psb, pst, off,
                            eps, qw, kw, qsh, ksh, *dq, *dk, dqw, dkw, ws, wsn, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), pn.EINVAL), (dict(dtype=-1), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(hk=-2), pn.EINVAL),
    (dict(D=0), pn.EUNSUPPORTED), (dict(D=257), pn.EUNSUPPORTED), (dict(R=3), pn.EINVAL), (dict(R=10), pn.EINVAL),
    (dict(inter=2), pn.EINVAL), (dict(hq=0, hk=1), pn.EINVAL), (dict(q=TOK(0)), pn.EINVAL),
    (dict(q=(4 * GIB + 2, 64, 32, 8)), pn.EINVAL), (dict(q=TOK(4, sb=-1)), pn.EINVAL), (dict(qo=0), pn.EINVAL),
    (dict(ko=0), pn.EINVAL), (dict(table=0), pn.EINVAL), (dict(n_pos=-1), pn.EINVAL), (dict(pos=12 * GIB, pos64=2), pn.EINVAL),
    (dict(pos=12 * GIB + 4, pos64=1), pn.EINVAL), (dict(B=1 << 20, T=1 << 20), pn.EUNSUPPORTED),
    (dict(qo=5 * GIB), pn.EINVAL), (dict(qo=7 * GIB), pn.EINVAL), (dict(ko=8 * GIB), pn.EINVAL),
    (dict(qo=4 * GIB + 4), pn.EINVAL), (dict(q=TOK(4, sh=16), qo=4 * GIB), pn.EINVAL),
    (dict(pos=12 * GIB, pst=1, psb=1 << 41), pn.EINVAL)])
def test_rotary_refusals(kw, code):
    for name in ("pn_rotary", "pn_qk_norm_rotary", "pn_qk_norm_rotary_backward"):
        assert getattr(pn.lib(), name)(_rotary_block(**kw)) == code, name
        assert pn.last_error() != ""


@pytest.mark.parametrize("kw, code", [
    (dict(eps=-1.0), pn.EINVAL), (dict(eps=float("nan")), pn.EINVAL), (dict(eps=float("inf")), pn.EINVAL),
    (dict(qw=12 * GIB, qsh=4), pn.EINVAL), (dict(kw=12 * GIB, ksh=-8), pn.EINVAL), (dict(qw=12 * GIB + 2), pn.EINVAL)])
def test_norm_refusals(kw, code):
    for name in ("pn_qk_norm_rotary", "pn_qk_norm_rotary_backward"):
        assert getattr(pn.lib(), name)(_rotary_block(**kw)) == code, name
    assert pn.lib().pn_qk_norm_rotary_workspace_bytes(_rotary_block(eps=-1.0)) == 0


def test_norm_backward_refusals():
    f = pn.lib().pn_qk_norm_rotary_backward
    n = pn.lib().pn_qk_norm_rotary_workspace_bytes(_rotary_block())
    assert n > 0
    assert f(_rotary_block()) == pn.EWORKSPACE                                    # none
    assert f(_rotary_block(ws=13 * GIB, wsn=n - 1)) == pn.EWORKSPACE               # too small
    assert f(_rotary_block(ws=13 * GIB + 8, wsn=n + 256)) == pn.EWORKSPACE         # misaligned
    assert f(_rotary_block(dq=TOK(0))) == pn.EINVAL
    assert f(_rotary_block(qo=4 * GIB)) == pn.EINVAL                              # not in place
    assert f(_rotary_block(qo=9 * GIB)) == pn.EINVAL
    assert f(_rotary_block(qw=12 * GIB, dqw=6 * GIB)) == pn.EINVAL
    assert f(_rotary_block(qw=12 * GIB, kw=12 * GIB, dqw=14 * GIB, dkw=14 * GIB)) == pn.EINVAL


def test_empty_problems_return_before_device_work():
    for kw in (dict(B=0), dict(T=0), dict(hq=0, hk=0)):
        for name in ("pn_rotary", "pn_qk_norm_rotary", "pn_qk_norm_rotary_backward"):
            assert getattr(pn.lib(), name)(_rotary_block(**kw)) == pn.OK
    for kw in (dict(B=0), dict(H=0, HK=1)):
        assert pn.lib().pn_linear_attention(_attention_block(**kw)) == pn.OK
        assert pn.lib().pn_linear_attention_backward(_attention_block(**kw)) == pn.OK
    assert pn.lib().pn_linear_attention_step(_step_block(B=0)) == pn.OK


def test_null_arguments():
    for name in ("pn_rotary", "pn_qk_norm_rotary", "pn_qk_norm_rotary_backward", "pn_linear_attention",
                 "pn_linear_attention_backward", "pn_linear_attention_step"):
        assert getattr(pn.lib(), name)(None) == pn.EINVAL
    assert pn.lib().pn_linear_attention_workspace_bytes(None, 0) == 0
    assert pn.lib().pn_qk_norm_rotary_workspace_bytes(None) == 0


def test_rotary_table_refusals():
    import ctypes
    f = pn.lib().pn_rotary_table
    one = (ctypes.c_double * 1)(1.0)
    assert f(None, 1, 4, 1.0, GIB, None) == pn.EINVAL
    assert f(one, 0, 4, 1.0, GIB, None) == pn.EUNSUPPORTED
    assert f((ctypes.c_double * 129)(), 129, 4, 1.0, GIB, None) == pn.EUNSUPPORTED
    assert f(one, 1, -1, 1.0, GIB, None) == pn.EINVAL
    assert f((ctypes.c_double * 1)(float("nan")), 1, 4, 1.0, GIB, None) == pn.EINVAL
    assert f(one, 1, 4, float("inf"), GIB, None) == pn.EINVAL
    assert f(one, 1, 4, 1.0, None, None) == pn.EINVAL
    assert f(one, 1, 0, 1.0, None, None) == pn.OK


def _attention_block(dtype=0, B=2, T=2, H=4, HK=4, dk=8, dv=8, scale=1.0, g=3 * GIB, lengths=0, q=TOK(4), k=TOK(5), v=TOK(6),
                     s0=0, o=7 * GIB, final=0, do=TOK(8), dfin=0, dq=9 * GIB, dk_=10 * GIB, dv_=11 * GIB, d0=0, ws=0, wsn=0):
    return seq._ATTENTION(dtype, B, T, H, HK, dk, dv, scale, g, lengths, *q, *k, *v, s0, o, final, *do, dfin, dq, dk_, dv_,
                               d0, ws, wsn, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(HK=3), pn.EINVAL), (dict(HK=0), pn.EINVAL),
    (dict(dk=0), pn.EUNSUPPORTED), (dict(dv=257), pn.EUNSUPPORTED), (dict(scale=float("nan")), pn.EINVAL),
    (dict(g=0), pn.EINVAL), (dict(q=TOK(0)), pn.EINVAL), (dict(k=TOK(5, st=-1)), pn.EINVAL),
    (dict(v=(6 * GIB + 1, 64, 32, 8)), pn.EINVAL), (dict(g=3 * GIB + 2), pn.EINVAL), (dict(lengths=12 * GIB + 1), pn.EINVAL),
    (dict(T=1 << 31), pn.EUNSUPPORTED), (dict(B=1 << 20, H=32, HK=1), pn.EUNSUPPORTED)])
def test_attention_refusals(kw, code):
    assert pn.lib().pn_linear_attention(_attention_block(**kw)) == code
    assert pn.lib().pn_linear_attention_backward(_attention_block(**kw)) == code
    assert pn.last_error() != ""


def test_attention_output_and_workspace_refusals():
    f, b = pn.lib().pn_linear_attention, pn.lib().pn_linear_attention_backward
    n = pn.lib().pn_linear_attention_workspace_bytes
    for kw in (dict(o=0), dict(o=4 * GIB), dict(o=7 * GIB + 2), dict(s0=12 * GIB, final=12 * GIB), dict(final=7 * GIB),
               dict(final=3 * GIB)):
        assert f(_attention_block(**kw)) == pn.EINVAL, kw
    for kw in (dict(dq=0), dict(dk_=9 * GIB), dict(dv_=8 * GIB), dict(do=TOK(0)), dict(d0=12 * GIB, s0=12 * GIB),
               dict(d0=12 * GIB, dfin=12 * GIB)):
        assert b(_attention_block(**kw)) == pn.EINVAL, kw
    big = dict(H=4, HK=2, T=4096, q=TOK(4, 1 << 20, 32, 8), k=TOK(5, 1 << 20, 16, 8), v=TOK(6, 1 << 20, 16, 8),
               do=TOK(8, 1 << 20, 32, 8))
    need = n(_attention_block(**big), 1)
    assert need > 256                                    # shared heads: float32 dk and dv of each head, at least
    assert b(_attention_block(**big)) == pn.EWORKSPACE
    assert b(_attention_block(**big, ws=20 * GIB, wsn=need - 1)) == pn.EWORKSPACE
    assert b(_attention_block(**big, ws=20 * GIB + 128, wsn=need + 256)) == pn.EWORKSPACE
    assert b(_attention_block(**big, ws=9 * GIB, wsn=need)) == pn.EINVAL
    assert n(_attention_block(HK=3), 0) == 0 and pn.last_error() != ""


def _step_block(dtype=0, B=2, H=4, HK=4, dk=8, dv=8, scale=1.0, g=3 * GIB, q=TOK(4), k=TOK(5), v=TOK(6), state=7 * GIB, slots=0,
                n_slots=2, o=9 * GIB):
    return seq._STEP(dtype, B, H, HK, dk, dv, scale, g, *q, *k, *v, state, slots, n_slots, o, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=7), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(HK=3), pn.EINVAL), (dict(dk=300), pn.EUNSUPPORTED),
    (dict(scale=float("inf")), pn.EINVAL), (dict(n_slots=-1), pn.EINVAL), (dict(n_slots=1), pn.EINVAL), (dict(g=0), pn.EINVAL),
    (dict(o=0), pn.EINVAL), (dict(state=0), pn.EINVAL), (dict(o=7 * GIB), pn.EINVAL), (dict(o=4 * GIB), pn.EINVAL),
    (dict(state=6 * GIB), pn.EINVAL), (dict(slots=10 * GIB + 2), pn.EINVAL), (dict(q=TOK(0)), pn.EINVAL)])
def test_step_refusals(kw, code):
    assert pn.lib().pn_linear_attention_step(_step_block(**kw)) == code
    assert pn.last_error() != ""


def test_binding_refuses_host_tensors_and_types():
    x = torch.zeros(1, 2, 3, 4)
    with pytest.raises(TypeError):
        pn.rotary(x, torch.zeros(4, 2, 2))
    with pytest.raises(TypeError):
        pn.linear_attention(x, x, x, torch.zeros(3))
    with pytest.raises(TypeError):
        pn.qk_norm_rotary(x, x, None, None, torch.zeros(4, 2, 2))
    with pytest.raises(TypeError):
        pn.linear_attention_step(x[:, 0], x[:, 0], x[:, 0], torch.zeros(3), x)
    with pytest.raises(ValueError):
        pn.rotary_table(4, [1.0], device="cpu")
