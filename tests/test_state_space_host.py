"""State-space operators without a GPU: the float64 oracle against differences and independent forms, and the C entries'
refusals (placeholder addresses; nothing is dereferenced)."""

import numpy as np
import pytest
import torch

import newton_evaluation_nonlinear_amd as pn
from newton_evaluation_nonlinear_amd import state_space as ss
from oracle import state_space as ref


@pytest.fixture(autouse=True)
def _no_error_left():
    yield
    pn.lib().pn_short_conv(_conv(B=0))                   # a call that succeeds clears the thread's message


def _rng(seed=0):
    return np.random.default_rng(seed)


def _differences(f, arrays, grads, tol=1e-7, h=1e-6):
    """Every element of the gradients against central differences of f(arrays)."""
    for name, g in grads.items():
        for i in np.ndindex(arrays[name].shape):
            values = []
            for d in (h, -h):
                moved = {**arrays, name: arrays[name].copy()}
                moved[name][i] += d
                values.append(f(moved))
            d = (values[0] - values[1]) / (2 * h)
            assert abs(d - g[i]) < tol * max(1.0, abs(d)) + tol, (name, i, d, g[i])


# ---------------------------------------------------------------- oracle pins


def test_conv_is_torchs_convolution():
    g = _rng(1)
    B, T, D, W = 2, 9, 5, 4
    x, w, bias, past = g.standard_normal((B, T, D)), g.standard_normal((D, W)), g.standard_normal(D), g.standard_normal((B, W - 1, D))
    y, final, _ = ref.short_conv(x, w, bias, past)
    rows = torch.tensor(np.concatenate((past, x), 1)).transpose(1, 2)
    want = torch.nn.functional.silu(torch.nn.functional.conv1d(rows, torch.tensor(w)[:, None], torch.tensor(bias), groups=D))
    assert np.allclose(y, want.transpose(1, 2).numpy(), atol=1e-12) and np.array_equal(final, x[:, T - W + 1:])


@pytest.mark.parametrize("activation", [True, False])
def test_conv_gradient_against_differences(activation):
    g = _rng(2)
    B, T, D, W = 2, 5, 3, 4
    a = dict(x=g.standard_normal((B, T, D)), w=g.standard_normal((D, W)), bias=g.standard_normal(D), s0=g.standard_normal((B, W - 1, D)))
    n, dy, df = [5, 2], g.standard_normal((B, T, D)), g.standard_normal((B, W - 1, D))

    def loss(a):
        y, s, _ = ref.short_conv(a["x"], a["w"], a["bias"], a["s0"], n, activation)
        return float((y * dy).sum() + (s * df).sum())

    grads, mags = ref.short_conv_backward(dy, a["x"], a["w"], a["bias"], a["s0"], df, n, activation)
    _differences(loss, a, dict(zip(("x", "w", "bias", "s0"), grads)))
    assert all((m >= np.abs(v) - 1e-12).all() for v, m in zip(grads, mags))


def test_scan_is_the_sum_over_earlier_tokens():
    g = _rng(3)
    B, T, D, G, N = 2, 7, 4, 2, 3
    x, dt, z = (g.standard_normal((B, T, D)) for _ in range(3))
    b, c = g.standard_normal((B, T, G, N)), g.standard_normal((B, T, G, N))
    A, skip, bias, h0 = -np.exp(g.standard_normal((D, N))), g.standard_normal(D), g.standard_normal(D), g.standard_normal((B, D, N))
    n = [7, 4]
    y, h = ref.ssm_scan(x, dt, A, b, c, skip, z, bias, True, h0, n)
    delta = np.log(1 + np.exp(dt + bias))
    for i in range(B):
        for d in range(D):
            k = d // 2
            S = np.cumsum(delta[i, :, d])
            for t in range(n[i]):
                state = np.exp(A[d] * S[t]) * h0[i, d]
                for s in range(t + 1):
                    state = state + np.exp(A[d] * (S[t] - S[s])) * delta[i, s, d] * x[i, s, d] * b[i, s, k]
                want = (state @ c[i, t, k] + skip[d] * x[i, t, d]) * z[i, t, d] / (1 + np.exp(-z[i, t, d]))
                assert abs(y[i, t, d] - want) < 1e-12
            assert np.allclose(h[i, d], state, atol=1e-12)
    assert not y[1, 4:].any()


@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradient_against_differences(softplus):
    g = _rng(4)
    B, T, D, G, N = 2, 4, 4, 2, 2
    a = dict(x=g.standard_normal((B, T, D)), dt=g.standard_normal((B, T, D)), A=-np.exp(g.standard_normal((D, N))),
             b=g.standard_normal((B, T, G, N)), c=g.standard_normal((B, T, G, N)), skip=g.standard_normal(D),
             z=g.standard_normal((B, T, D)), bias=g.standard_normal(D), h0=g.standard_normal((B, D, N)))
    n, dy, dh = [4, 3], g.standard_normal((B, T, D)), g.standard_normal((B, D, N))

    def loss(a):
        y, h = ref.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"], a["skip"], a["z"], a["bias"], softplus, a["h0"], n)
        return float((y * dy).sum() + (h * dh).sum())

    args = (a["x"], a["dt"], a["A"], a["b"], a["c"], a["skip"], a["z"], a["bias"], softplus, a["h0"])
    grads = ref.ssm_scan_backward(dy, *args, dh, n)
    names = ("x", "dt", "A", "b", "c", "skip", "z", "bias", "h0")
    _differences(loss, a, dict(zip(names, grads)), tol=2e-7)
    bounds = ref.ssm_scan_backward(dy, *args, dh, n, bound=True)
    assert all((m >= np.abs(v) - 1e-12).all() for v, m in zip(grads, bounds))


@pytest.mark.parametrize("drop", [(), ("gate",), ("post_weight",), ("scale",), ("weight",), ("gate", "post_weight", "scale"),
                                  ("residual",), ("residual", "post_weight")])
def test_norm_gradient_against_differences(drop):
    g = _rng(5)
    a = dict(x=g.standard_normal((2, 3, 5)), residual=g.standard_normal((2, 3, 5)), gate=g.standard_normal((2, 3, 5)),
             weight=g.standard_normal(5), post_weight=g.standard_normal(5), scale=g.standard_normal(5))
    a = {k: v for k, v in a.items() if k not in drop}
    dy, ds, eps = g.standard_normal((2, 3, 5)), g.standard_normal((2, 3, 5)), 1e-3

    def loss(a):
        y, s = ref.block_norm(**a, eps=eps)
        return float((0.0 if y is None else (y * dy).sum()) + (s * ds).sum())

    grads, mags = ref.block_norm_backward(dy, ds, **a, eps=eps)
    named = dict(zip(("x", "weight", "residual", "gate", "post_weight", "scale"), grads))
    assert all((v is None) == (k not in a) for k, v in named.items())
    _differences(loss, a, {k: v for k, v in named.items() if v is not None})
    assert all(v is None or (m >= np.abs(v) - 1e-12).all() for v, m in zip(grads, mags))


# ---------------------------------------------------------------- refusals of the C entries

GIB = 1 << 30
TOK = lambda i, sb=64, st=32, sh=0: (i * GIB, sb, st, sh)  # noqa: E731


def _conv(dtype=0, B=2, T=2, D=8, W=4, act=1, w=3 * GIB, bias=0, n=0, x=TOK(4), s0=0, y=6 * GIB, final=0, dy=TOK(7), df=0,
          dx=8 * GIB, dw=9 * GIB, db=0, d0=0, ws=0, wsn=0):
    return ss._CONV(dtype, B, T, D, W, act, w, bias, n, *x, s0, y, final, *dy, df, dx, dw, db, d0, ws, wsn, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(T=-2), pn.EINVAL), (dict(W=0), pn.EUNSUPPORTED),
    (dict(W=9), pn.EUNSUPPORTED), (dict(act=2), pn.EINVAL), (dict(w=0), pn.EINVAL), (dict(w=3 * GIB + 2), pn.EINVAL),
    (dict(n=5 * GIB + 1), pn.EINVAL), (dict(x=TOK(0)), pn.EINVAL), (dict(x=TOK(4, sb=-1)), pn.EINVAL),
    (dict(x=(4 * GIB + 2, 64, 32, 0)), pn.EINVAL), (dict(s0=5 * GIB + 2), pn.EINVAL), (dict(B=1 << 20, T=1 << 20), pn.EUNSUPPORTED),
    (dict(T=1 << 31), pn.EUNSUPPORTED), (dict(x=TOK(4, st=1 << 41)), pn.EINVAL)])
def test_conv_refusals(kw, code):
    need = pn.lib().pn_short_conv_workspace_bytes(_conv())
    assert need > 256
    assert pn.lib().pn_short_conv(_conv(**kw)) == code
    assert pn.last_error() != ""
    assert pn.lib().pn_short_conv_backward(_conv(ws=20 * GIB, wsn=need, **kw)) == code


def test_conv_outputs_and_workspace():
    f, b = pn.lib().pn_short_conv, pn.lib().pn_short_conv_backward
    for kw in (dict(y=0), dict(y=4 * GIB), dict(y=3 * GIB), dict(final=6 * GIB), dict(s0=5 * GIB, final=5 * GIB), dict(y=6 * GIB + 2)):
        assert f(_conv(**kw)) == pn.EINVAL, kw
    n = pn.lib().pn_short_conv_workspace_bytes(_conv())
    assert b(_conv()) == b(_conv(ws=20 * GIB, wsn=n - 1)) == b(_conv(ws=20 * GIB + 8, wsn=n)) == pn.EWORKSPACE
    ok = dict(ws=20 * GIB, wsn=n)
    for kw in (dict(dx=0), dict(dw=0), dict(bias=10 * GIB), dict(dx=4 * GIB), dict(dx=7 * GIB), dict(dw=8 * GIB), dict(dy=TOK(0)),
               dict(d0=8 * GIB), dict(df=11 * GIB, d0=11 * GIB)):
        assert b(_conv(**{**ok, **kw})) == pn.EINVAL, kw
    assert b(_conv(ws=8 * GIB, wsn=n)) == pn.EINVAL
    assert pn.lib().pn_short_conv_workspace_bytes(_conv(W=9)) == 0 and pn.last_error() != ""
    assert pn.lib().pn_short_conv_workspace_bytes(_conv(B=0)) == 256


def _conv_step(dtype=0, B=2, D=8, W=4, act=1, w=3 * GIB, bias=0, x=TOK(4), state=5 * GIB, slots=0, n_slots=2, y=6 * GIB):
    return ss._CONV_STEP(dtype, B, D, W, act, w, bias, *x, state, slots, n_slots, y, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=-1), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(W=9), pn.EUNSUPPORTED), (dict(w=0), pn.EINVAL), (dict(y=0), pn.EINVAL),
    (dict(state=0), pn.EINVAL), (dict(n_slots=1), pn.EINVAL), (dict(n_slots=-1), pn.EINVAL), (dict(slots=7 * GIB + 2), pn.EINVAL),
    (dict(y=4 * GIB), pn.EINVAL), (dict(y=5 * GIB), pn.EINVAL), (dict(state=4 * GIB), pn.EINVAL), (dict(x=TOK(0)), pn.EINVAL),
    (dict(n_slots=1 << 31, D=1 << 20), pn.EUNSUPPORTED)])
def test_conv_step_refusals(kw, code):
    assert pn.lib().pn_short_conv_step(_conv_step(**kw)) == code
    assert pn.last_error() != ""


BC = lambda i, sb=64, st=32, sh=16: (i * GIB, sb, st, sh)  # noqa: E731


def _scan(dtype=0, B=2, T=2, D=8, N=16, G=1, soft=1, A=3 * GIB, skip=0, bias=0, n=0, x=TOK(4), dt=TOK(5), z=TOK(0), b=BC(6), c=BC(7),
          s0=0, y=8 * GIB, final=0, dy=TOK(9), df=0, dx=10 * GIB, ddt=11 * GIB, dz=0, db=12 * GIB, dc=13 * GIB, dA=14 * GIB, dskip=0,
          dbias=0, d0=0, ws=0, wsn=0):
    return ss._SSM(dtype, B, T, D, N, G, soft, A, skip, bias, n, *x, *dt, *z, *b, *c, s0, y, final, *dy, df, dx, ddt, dz, db, dc, dA,
                   dskip, dbias, d0, ws, wsn, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(N=0), pn.EUNSUPPORTED), (dict(N=129), pn.EUNSUPPORTED),
    (dict(G=0), pn.EINVAL), (dict(G=3), pn.EINVAL), (dict(G=16), pn.EINVAL), (dict(soft=2), pn.EINVAL), (dict(A=0), pn.EINVAL),
    (dict(A=3 * GIB + 2), pn.EINVAL), (dict(x=TOK(0)), pn.EINVAL), (dict(dt=TOK(0)), pn.EINVAL), (dict(b=BC(0)), pn.EINVAL),
    (dict(c=(7 * GIB + 1, 64, 32, 16)), pn.EINVAL), (dict(z=(15 * GIB + 2, 64, 32, 0), dz=16 * GIB), pn.EINVAL),
    (dict(b=BC(6, sh=-1)), pn.EINVAL), (dict(n=17 * GIB + 2), pn.EINVAL), (dict(T=1 << 31), pn.EUNSUPPORTED),
    (dict(B=1 << 20, T=1 << 10, D=1 << 12), pn.EUNSUPPORTED), (dict(D=1 << 25), pn.EUNSUPPORTED),
    (dict(x=TOK(4, st=(1 << 26) + 1)), pn.EUNSUPPORTED), (dict(b=BC(6, st=1 << 27)), pn.EUNSUPPORTED)])
def test_scan_refusals(kw, code):
    need = pn.lib().pn_ssm_scan_workspace_bytes(_scan(), 1)
    assert need > 256
    assert pn.lib().pn_ssm_scan(_scan(**kw)) == code
    assert pn.last_error() != ""
    assert pn.lib().pn_ssm_scan_backward(_scan(ws=40 * GIB, wsn=need, **kw)) == code


def test_scan_outputs_and_workspace():
    f, b = pn.lib().pn_ssm_scan, pn.lib().pn_ssm_scan_backward
    size = pn.lib().pn_ssm_scan_workspace_bytes
    for kw in (dict(y=0), dict(y=4 * GIB), dict(y=7 * GIB), dict(y=3 * GIB), dict(final=8 * GIB), dict(s0=18 * GIB, final=18 * GIB)):
        assert f(_scan(**kw)) == pn.EINVAL, kw
    assert size(_scan(), 0) == 256                       # one segment
    long = dict(T=4096, x=TOK(4, 1 << 20), dt=TOK(5, 1 << 20), b=BC(6, 1 << 20), c=BC(7, 1 << 20), dy=TOK(9, 1 << 20))
    need = size(_scan(**long), 0)
    assert need > 256
    assert f(_scan(**long)) == f(_scan(**long, ws=40 * GIB, wsn=need - 1)) == f(_scan(**long, ws=40 * GIB + 64, wsn=need)) == pn.EWORKSPACE
    assert f(_scan(**long, ws=8 * GIB, wsn=need)) == pn.EINVAL
    n = size(_scan(), 1)
    ok = dict(ws=40 * GIB, wsn=n)
    for kw in (dict(dx=0), dict(ddt=0), dict(db=0), dict(dc=0), dict(dA=0), dict(skip=18 * GIB), dict(bias=18 * GIB),
               dict(z=TOK(18)), dict(dx=11 * GIB), dict(dx=4 * GIB), dict(db=9 * GIB), dict(dy=TOK(0)), dict(d0=14 * GIB),
               dict(df=19 * GIB, d0=19 * GIB)):
        assert b(_scan(**{**ok, **kw})) == pn.EINVAL, kw
    assert size(_scan(N=129), 0) == 0 and pn.last_error() != ""
    assert size(_scan(B=0), 1) == 256


@pytest.mark.parametrize("N", [1, 8, 16, 17, 128])
def test_scan_workspace_at_every_small_length(N):
    """A size for every length, that does not shrink with it while there is one segment, and none for a forward call of one."""
    size = pn.lib().pn_ssm_scan_workspace_bytes
    for B, D in ((1, 1), (1, 33), (3, 300), (64, 1100), (2000, 40)):
        last = 0
        for T in range(200):
            n, back = size(_scan(B=B, T=T, D=D, N=N), 0), size(_scan(B=B, T=T, D=D, N=N), 1)
            assert n >= 256 and back > 256 and (T >= 64 or n == 256), (B, D, T)
            assert T >= 24 or back >= last
            last = back


def _scan_step(dtype=0, B=2, D=8, N=16, G=1, soft=1, A=3 * GIB, skip=0, bias=0, x=TOK(4), dt=TOK(5), z=TOK(0), b=BC(6), c=BC(7),
               state=8 * GIB, slots=0, n_slots=2, y=9 * GIB):
    return ss._SSM_STEP(dtype, B, D, N, G, soft, A, skip, bias, *x, *dt, *z, *b, *c, state, slots, n_slots, y, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=9), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(N=200), pn.EUNSUPPORTED), (dict(G=5), pn.EINVAL), (dict(A=0), pn.EINVAL),
    (dict(y=0), pn.EINVAL), (dict(state=0), pn.EINVAL), (dict(n_slots=1), pn.EINVAL), (dict(n_slots=-1), pn.EINVAL),
    (dict(slots=10 * GIB + 2), pn.EINVAL), (dict(y=8 * GIB), pn.EINVAL), (dict(y=4 * GIB), pn.EINVAL), (dict(state=7 * GIB), pn.EINVAL),
    (dict(dt=TOK(0)), pn.EINVAL), (dict(b=BC(6, sb=-3)), pn.EINVAL),
    (dict(n_slots=1 << 31, D=1 << 20), pn.EUNSUPPORTED), (dict(B=1 << 20, D=1 << 16), pn.EUNSUPPORTED)])
def test_scan_step_refusals(kw, code):
    assert pn.lib().pn_ssm_step(_scan_step(**kw)) == code
    assert pn.last_error() != ""


def _norm(dtype=1, rdtype=0, B=2, T=2, D=8, eps=1e-6, w=3 * GIB, pw=4 * GIB, sc=5 * GIB, x=TOK(6), z=TOK(7), r=TOK(8), y=9 * GIB,
          s=10 * GIB, dy=TOK(11), ds=TOK(12), dx=14 * GIB, dz=15 * GIB, dr=16 * GIB, dw=17 * GIB, dpw=18 * GIB,
          dsc=19 * GIB, ws=0, wsn=0):
    return ss._NORM(dtype, rdtype, B, T, D, eps, w, pw, sc, *x, *z, *r, y, s, *dy, *ds, dx, dz, dr, dw, dpw, dsc, ws, wsn, 0)


@pytest.mark.parametrize("kw, code", [
    (dict(dtype=3), pn.EINVAL), (dict(rdtype=2), pn.EINVAL), (dict(B=-1), pn.EINVAL), (dict(D=0), pn.EUNSUPPORTED),
    (dict(D=8193), pn.EUNSUPPORTED), (dict(eps=-1.0), pn.EINVAL), (dict(eps=float("nan")), pn.EINVAL), (dict(w=3 * GIB + 2), pn.EINVAL),
    (dict(x=TOK(0)), pn.EINVAL), (dict(z=(7 * GIB + 1, 64, 32, 0)), pn.EINVAL), (dict(x=TOK(6, st=-8)), pn.EINVAL)])
def test_norm_refusals(kw, code):
    need = pn.lib().pn_block_norm_workspace_bytes(_norm())
    assert need > 256
    assert pn.lib().pn_block_norm(_norm(**kw)) == code
    assert pn.last_error() != ""
    assert pn.lib().pn_block_norm_backward(_norm(ws=40 * GIB, wsn=need, **kw)) == code


def test_norm_outputs_and_workspace():
    f, b = pn.lib().pn_block_norm, pn.lib().pn_block_norm_backward
    for kw in (dict(y=0), dict(s=0), dict(y=10 * GIB), dict(y=6 * GIB), dict(s=8 * GIB), dict(s=10 * GIB + 2), dict(r=(8 * GIB + 2, 64, 32, 0))):
        assert f(_norm(**kw)) == pn.EINVAL, kw
    n = pn.lib().pn_block_norm_workspace_bytes(_norm())
    assert b(_norm()) == b(_norm(ws=40 * GIB, wsn=n - 1)) == b(_norm(ws=40 * GIB + 8, wsn=n)) == pn.EWORKSPACE
    ok = dict(ws=40 * GIB, wsn=n)
    for kw in (dict(dx=0), dict(dz=0), dict(dw=0), dict(dpw=0), dict(dsc=0), dict(dy=TOK(0)), dict(dx=6 * GIB),
               dict(dr=8 * GIB), dict(dr=12 * GIB), dict(dz=14 * GIB), dict(dr=16 * GIB + 2)):
        assert b(_norm(**{**ok, **kw})) == pn.EINVAL, kw
    assert pn.lib().pn_block_norm_workspace_bytes(_norm(w=0, pw=0, sc=0)) == 256
    assert pn.lib().pn_block_norm_workspace_bytes(_norm(D=0)) == 0 and pn.last_error() != ""


ENTRIES = [n for n in ss.EXPORTED if not n.endswith("_bytes")]


@pytest.mark.parametrize("name", ENTRIES)
def test_null_arguments(name):
    assert getattr(pn.lib(), name)(None) == pn.EINVAL
    assert pn.lib().pn_ssm_scan_workspace_bytes(None, 0) == pn.lib().pn_short_conv_workspace_bytes(None) == 0
    assert pn.lib().pn_block_norm_workspace_bytes(None) == 0


def test_empty_problems_return_before_device_work():
    L = pn.lib()
    for kw in (dict(B=0), dict(D=0)):
        assert L.pn_short_conv(_conv(**kw)) == L.pn_short_conv_step(_conv_step(**kw)) == pn.OK
        assert L.pn_ssm_scan(_scan(**kw)) == L.pn_ssm_step(_scan_step(**kw)) == pn.OK
    assert L.pn_short_conv_backward(_conv(D=0)) == L.pn_ssm_scan_backward(_scan(D=0)) == pn.OK
    for kw in (dict(B=0), dict(T=0)):
        assert L.pn_block_norm(_norm(**kw)) == pn.OK


def test_binding_refuses_host_tensors_and_types():
    x, w = torch.zeros(1, 2, 3), torch.zeros(3, 4)
    for call in (lambda: pn.short_conv(x, w), lambda: pn.short_conv_backward(x, x, w), lambda: pn.short_conv_step(x[0], w, x),
                 lambda: pn.ssm_scan(x, x, w, x[..., None], x[..., None]), lambda: pn.ssm_step(x[0], x[0], w, x, x, x),
                 lambda: pn.ssm_scan_backward(x, x, x, w, x, x), lambda: pn.block_norm(x), lambda: pn.block_norm_backward(x, x, x, x),
                 lambda: pn.short_conv("x", w), lambda: pn.block_norm(None)):
        with pytest.raises(TypeError):
            call()
