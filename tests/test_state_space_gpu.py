"""State-space operators on the GPU against the float64 oracle.

Tolerances.  U is 2^-24 and u the unit roundoff of the storage type (2^-24, 2^-8, 2^-11), added once to every stored result.
The convolution and the norms: the error of each function used (below), and n roundings of sums of n terms, relative to the
sums of the absolute values of their terms.  The scan: a running error bound (`scan_bounds`) that goes through the recurrence
as the kernels do, with the roundings of every product and sum.

The functions: e^v by an exponential to base two with the argument rounded twice: (2 |v| + 2) U of it; so v sigmoid(v) is
within (2 |v| + 8) U of itself, its slope p (1 + v (1 - p)) within p (1 + |v|) (2 |v| + 10) U, and
softplus(v) within (3 |v| + 8) U of itself.
"""

import numpy as np
import pytest
import torch

import newton_evaluation_nonlinear_amd as pn
from oracle import state_space as ref
from test_sequence_gpu import DEV, ROUND, TINY, TYPES, _np, _rand
from test_sequence_gpu import _close as _within

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _n(t):
    return None if t is None else _np(t)


def _lengths(n):
    return None if n is None else torch.tensor(n, dtype=torch.int32, device=DEV)


def _close(got, want, bound, what):
    """Within the bound; a value that rounds past binary16's largest, 65504 (from 65520 on), is an infinity of its sign."""
    if got.dtype is torch.float16:
        x = _np(got)
        over = np.isinf(x) & (np.sign(x) == np.sign(want)) & (np.abs(want) + bound >= 65520.0)
        want = np.where(over, 0.0, want)
        got = torch.where(torch.from_numpy(over).to(got.device), torch.zeros_like(got), got)
    _within(got, want, bound, what)


def _bound(dtype, want, err):
    return ROUND[dtype] * np.abs(want) + 1.01 * err + TINY[dtype]


# ---------------------------------------------------------------- short convolution


def conv_inputs(dtype, B, T, D, W, initial, seed=0):
    g = torch.Generator().manual_seed(seed)
    return dict(x=_rand(g, (B, T, D), dtype), weight=_rand(g, (D, W), "f32", 0.6), bias=_rand(g, (D,), "f32", 0.5),
                initial_state=_rand(g, (B, W - 1, D), dtype) if initial else None, dy=_rand(g, (B, T, D), dtype),
                d_final_state=_rand(g, (B, W - 1, D), dtype, 0.5) if initial else None)


def check_conv(a, dtype, lengths=None, activation=True, backward=True):
    W = a["weight"].shape[1]
    print(f"[conv] {dtype} x{tuple(a['x'].shape)} W={W} lengths={lengths} act={activation} "
          f"initial={a['initial_state'] is not None}", flush=True)
    names = ("x", "weight", "bias", "initial_state")
    h = {k: _n(v) for k, v in a.items()}
    kw = dict(initial_state=a["initial_state"], bias=a["bias"], lengths=_lengths(lengths), activation=activation)
    y, final = pn.short_conv(a["x"], a["weight"], **kw)
    wy, wf, pre = ref.short_conv(*(h[k] for k in names), lengths, activation)
    mag = ref.short_conv(*(None if h[k] is None else np.abs(h[k]) for k in names), lengths, False)[0]
    err = (W + 2) * U * mag
    _close(y, wy, _bound(dtype, wy, 1.1 * err + (2 * np.abs(pre) + 8) * U * np.abs(wy)), "y")
    assert np.array_equal(_np(final), wf)
    if not backward:
        return
    got = pn.short_conv_backward(a["dy"], a["x"], a["weight"], d_final_state=a["d_final_state"], **kw)
    args = (h["weight"], h["bias"], h["initial_state"])
    want, mags = ref.short_conv_backward(h["dy"], h["x"], *args, h["d_final_state"], lengths, activation)
    # the error of d = dy act'(pre), |act''| <= 1/2, through the sums of the gradients of the plain convolution
    e = np.abs(h["dy"]) * ((0.5 * err + (1 + np.abs(pre)) * (2 * np.abs(pre) + 10) * U) if activation else U)
    through = ref.short_conv_backward(e, np.abs(h["x"]), np.abs(args[0]), None,
                                      None if args[2] is None else np.abs(args[2]), None, lengths, False)[0]
    for i, (x, name) in enumerate(zip(got, ("dx", "dweight", "dbias", "d initial"))):
        if name == "d initial" and h["initial_state"] is None:
            assert x is None
            continue
        n = W + 3 if name.startswith("d initial") or name == "dx" else 64 + 2       # runs of up to 64 tokens, then float64
        stored = "f32" if name in ("dweight", "dbias") else dtype
        _close(x, want[i], _bound(stored, want[i], through[i] + n * U * mags[i]), name)


CONV = [(1, 1, 1, 1), (2, 1, 5, 4), (1, 2, 8, 8), (3, 7, 16, 2), (2, 63, 33, 3), (2, 64, 64, 4), (1, 65, 40, 5), (1, 300, 24, 8),
        (2, 200, 130, 4), (4, 33, 512, 1), (1, 9, 4096, 4)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", CONV, ids=["x".join(map(str, s)) for s in CONV])
def test_conv_shapes(dtype, shape):
    for initial in (False, True):
        check_conv(conv_inputs(dtype, *shape, initial), dtype, activation=initial or shape[1] % 2 == 0)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [2, 4, 7])
def test_conv_lengths(dtype, W):
    """Sequences that end at every place of a run; padding is never read, and its rows are 0."""
    a = conv_inputs(dtype, 7, 130, 24, W, True)
    n = [0, 1, 2, W, 64, 65, 130]
    given = [-5, 1, 2, W, 64, 65, 100000]
    check_conv(a, dtype, lengths=n)
    dirty = {k: None if v is None else v.clone() for k, v in a.items()}
    for b, m in enumerate(n):
        dirty["x"][b, m:] = float("nan")
        dirty["dy"][b, m:] = float("inf")
    for f, first in ((pn.short_conv, ()), (pn.short_conv_backward, ("dy",))):
        more = dict(d_final_state=a["d_final_state"]) if first else {}
        got = [f(*[x[i] for i in first + ("x", "weight")], bias=a["bias"], initial_state=a["initial_state"], lengths=_lengths(m), **more)
               for x, m in ((dirty, given), (a, n))]
        for x, y in zip(*got):
            assert torch.equal(x, y) and bool(torch.isfinite(x).all())
    y, final = pn.short_conv(a["x"], a["weight"], initial_state=a["initial_state"], lengths=_lengths(given))
    assert torch.equal(final[0], a["initial_state"][0])
    for b, m in enumerate(n):
        assert not y[b, m:].any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_conv_strides(dtype):
    """Views of a packed projection, starts off any vector boundary, a broadcast batch, time before batch."""
    g = torch.Generator().manual_seed(2)
    a = conv_inputs(dtype, 2, 70, 40, 4, True)
    packed = _rand(g, (2, 70, 2 * 40 + 1), dtype)
    for x in (packed[..., 1:41], packed[..., 40:80], packed[:1, :, :40].expand(2, 70, 40),
              _rand(g, (70, 2, 40), dtype).transpose(0, 1)):
        check_conv(dict(a, x=x, dy=x.flip(1) if x.stride(0) else a["dy"]), dtype)


def test_conv_far_taps_do_not_touch_a_token():
    """A NaN or infinity reaches the W outputs that see it, whatever the width the kernel is built for."""
    for W in (1, 2, 3, 5, 6):
        for bad in (float("nan"), float("inf")):
            x = torch.randn(1, 40, 16, device=DEV)
            x[0, 13] = bad
            w = torch.ones(16, W, device=DEV)
            y, _ = pn.short_conv(x, w, activation=False)
            fine = torch.isfinite(y[0]).all(-1)
            assert [t for t in range(40) if not fine[t]] == list(range(13, 13 + W))
            dx, _, _, _ = pn.short_conv_backward(x, torch.randn(1, 40, 16, device=DEV), w, activation=False)
            fine = torch.isfinite(dx[0]).all(-1)
            assert [t for t in range(40) if not fine[t]] == list(range(13 - W + 1, 14))


def test_conv_without_tokens():
    a = conv_inputs("bf16", 2, 0, 24, 4, True)
    y, final = pn.short_conv(a["x"], a["weight"], initial_state=a["initial_state"])
    assert y.shape == (2, 0, 24) and torch.equal(final, a["initial_state"])
    assert not pn.short_conv(a["x"], a["weight"])[1].any()
    for d in (a["d_final_state"], None):
        dx, dw, db, d0 = pn.short_conv_backward(a["dy"], a["x"], a["weight"], bias=a["bias"], initial_state=a["initial_state"],
                                                d_final_state=d)
        assert torch.equal(d0, torch.zeros_like(d0) if d is None else d)
        assert not dw.any() and not db.any()
    empty = torch.empty(0, 5, 24, device=DEV)
    dx, dw, db, _ = pn.short_conv_backward(empty, empty, a["weight"], bias=a["bias"])
    assert not dw.any() and not db.any() and dx.shape == empty.shape


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [1, 3, 4, 5, 8])
def test_conv_many_sequences_are_the_few(dtype, W):
    """Where there are many sequences a thread takes longer runs of tokens: outputs and token gradients are those of a few
    sequences at a time, bit for bit.  The weights' gradients add at most 64 products in a run here, 16 there, then in 64 bits,
    and are rounded once: 82 roundings of the sum of magnitudes (which is off by 65 itself) and some to spare."""
    n = torch.randint(0, 262, (64,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    n[:4] = torch.tensor([0, 1, 64, 261])
    a = conv_inputs(dtype, 64, 261, 1024, W, True)
    a["lengths"] = n.to(DEV)

    def both(a, at):
        c = {k: v if k in ("weight", "bias") else v[at] for k, v in a.items()}
        kw = dict(bias=c["bias"], initial_state=c["initial_state"], lengths=c["lengths"])
        y = pn.short_conv(c["x"], c["weight"], **kw)
        return y, [pn.short_conv_backward(c["dy"], c["x"], c["weight"], d_final_state=c["d_final_state"], activation=act, **kw)
                   for act in (True, False)]

    y, grads = both(a, slice(None))
    mags = both({k: v if k == "lengths" else v.abs() for k, v in a.items()}, slice(None))[1][1]
    sums = [0.0, 0.0]
    for i in range(0, 64, 4):
        at = slice(i, i + 4)
        few, few_grads = both(a, at)
        assert torch.equal(y[0][at], few[0]) and torch.equal(y[1][at], few[1])
        for g, f in zip(grads, few_grads):
            assert torch.equal(g[0][at], f[0]) and torch.equal(g[3][at], f[3])
        sums = [s + t.double() for s, t in zip(sums, few_grads[1][1:3])]
    for got, want, mag in zip(grads[1][1:3], sums, mags[1:3]):
        assert bool(((got.double() - want).abs() <= 100 * 2.0 ** -24 * mag.double()).all())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("W", [1, 2, 4, 8])
@pytest.mark.parametrize("D", [24, 33])
def test_conv_steps_are_the_prompt(dtype, W, D):
    """Token by token through a pool, idle rows between, gives what the prompt gives, bit for bit."""
    a = conv_inputs(dtype, 3, 11, D, W, True)
    want, final = pn.short_conv(a["x"], a["weight"], bias=a["bias"], initial_state=a["initial_state"])
    pool = torch.full((6, W - 1, D), 7.0, dtype=TYPES[dtype], device=DEV)
    slots = torch.tensor([4, -1, 0, 2, 6], dtype=torch.int32, device=DEV)
    pool[[4, 0, 2]] = a["initial_state"]
    for t in range(11):
        x = torch.zeros(5, D, dtype=TYPES[dtype], device=DEV)
        x[[0, 2, 3]] = a["x"][:, t]
        y = pn.short_conv_step(x, a["weight"], pool, bias=a["bias"], slots=slots)
        assert torch.equal(y[[0, 2, 3]], want[:, t]) and not y[[1, 4]].any()
    assert torch.equal(pool[[4, 0, 2]], final) and bool((pool[[1, 3, 5]] == 7.0).all())


# ---------------------------------------------------------------- selective scan


def scan_inputs(dtype, B, T, D, N, G, initial=True, gate=True, seed=0, step=0.1):
    g = torch.Generator().manual_seed(seed)
    a = dict(x=_rand(g, (B, T, D), dtype), dt=_rand(g, (B, T, D), dtype, 0.5), b=_rand(g, (B, T, G, N), dtype),
             c=_rand(g, (B, T, G, N), dtype), dy=_rand(g, (B, T, D), dtype))
    a["A"] = -(torch.rand(D, N, generator=g) * 4 + 0.1).to(DEV)
    a["skip"] = _rand(g, (D,), "f32")
    a["dt_bias"] = (torch.rand(D, generator=g) * 3 + float(np.log(np.expm1(step))) - 1.5).to(DEV)
    a["gate"] = _rand(g, (B, T, D), dtype) if gate else None
    a["initial_state"] = _rand(g, (B, D, N), "f32") if initial else None
    a["d_final_state"] = _rand(g, (B, D, N), "f32", 0.5) if initial else None
    return a


def scan_bounds(h, lengths, use_softplus=True):
    """Bounds of the errors of (y, final state) and of the nine gradients, first order in U."""
    x, dt, A, dy = h["x"], h["dt"], h["A"], h["dy"]
    B, T, D = x.shape
    G, N = h["b"].shape[2:]
    raw = dt + (0.0 if h["dt_bias"] is None else h["dt_bias"])
    delta, slope = ref._steps(dt, h["dt_bias"], use_softplus)
    ab, ac = (np.abs(np.repeat(h[k], D // G, 2)) for k in "bc")
    skip = np.zeros(D) if h["skip"] is None else np.abs(h["skip"])
    eta = ((3 * np.abs(raw) + 8) if use_softplus else np.ones_like(raw)) * U
    join = lambda v: v.reshape(B, T, G, D // G, N).sum(3)  # noqa: E731
    ye, fe = np.zeros((B, T, D)), np.zeros((B, D, N))
    out = [np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((D, N)), np.zeros((B, T, D, N)), np.zeros((B, T, D, N)),
           np.zeros(D), np.zeros((B, T, D)), np.zeros(D), np.zeros((B, D, N))]
    dbm, dcm = np.zeros((B, T, D, N)), np.zeros((B, T, D, N))
    for i, n in enumerate(ref._lengths(lengths, B, T)):
        H = np.zeros((D, N)) if h["initial_state"] is None else np.abs(h["initial_state"][i])
        e, before, after, pre = np.zeros((D, N)), [], [], []
        a = np.exp(delta[i][..., None] * A)                                  # [T, D, N]
        # per step: the argument's error, also of sums of steps over a segment, and four roundings
        fade = np.abs(delta[i][..., None] * A) * (eta[i][..., None] + T * U) + 4 * U
        for t in range(n):
            K, Ke = a[t] * H, a[t] * (e + H * fade[t])
            before.append((K, Ke))
            ub = np.abs(delta[i, t] * x[i, t])[:, None] * ab[i, t]
            H = K + ub
            e = Ke + ub * (eta[i, t][:, None] + 3 * U) + 2 * U * H
            after.append((H, e))
            Y = (ac[i, t] * H).sum(-1) + skip * np.abs(x[i, t])
            Ye = (ac[i, t] * e).sum(-1) + (N + 6) * U * Y
            pre.append((Y, Ye))
            z = 0.0 if h["gate"] is None else h["gate"][i, t]
            Z = 1.0 if h["gate"] is None else np.abs(z * ref.logistic(z))
            ye[i, t] = Z * (Ye + Y * (2 * np.abs(z) + 8) * U)
        fe[i] = e + U * H
        r = np.zeros((D, N)) if h["d_final_state"] is None else np.abs(h["d_final_state"][i])
        re = np.zeros((D, N))
        for t in reversed(range(n)):
            z = np.zeros(D) if h["gate"] is None else h["gate"][i, t]
            p = ref.logistic(z)
            g = np.abs(dy[i, t]) * (1.0 if h["gate"] is None else np.abs(z * p))
            ge = g * (2 * np.abs(z) + 8) * U
            r = r + g[:, None] * ac[i, t]
            re = re + (ge + 2 * U * g)[:, None] * ac[i, t] + 2 * U * r
            (K, Ke), (H, He), (Y, Ye) = before[t], after[t], pre[t]
            du = (r * ab[i, t]).sum(-1)
            due = (re * ab[i, t]).sum(-1) + (N + 4) * U * du
            w, we = r * K, re * K + r * Ke + 3 * U * r * K
            dd = np.abs(x[i, t]) * du + (w * np.abs(A)).sum(-1)
            dde = np.abs(x[i, t]) * due + (we * np.abs(A)).sum(-1) + (N + 6) * U * dd
            d = np.abs(delta[i, t])
            out[0][i, t] = d * due + (eta[i, t] + 4 * U) * d * du + skip * ge + 4 * U * skip * g
            out[1][i, t] = slope[i, t] * (dde + dd * (2 * np.abs(raw[i, t]) + 8) * U)
            out[2] += we * d[:, None] + w * (d * (eta[i, t] + (T + 6) * U))[:, None]
            u = np.abs(delta[i, t] * x[i, t])[:, None]
            dbm[i, t], dcm[i, t] = r * u, g[:, None] * H
            out[3][i, t] = re * u + r * u * (eta[i, t] + 4 * U)[:, None]
            out[4][i, t] = ge[:, None] * H + g[:, None] * (He + 4 * U * H)
            out[5] += (ge + (T + 4) * U * g) * np.abs(x[i, t])
            if h["gate"] is not None:
                P = p * (1 + np.abs(z))
                out[6][i, t] = np.abs(dy[i, t]) * P * ((2 * np.abs(z) + 10) * U * Y + Ye)
            out[7] += out[1][i, t] + (T + 4) * U * slope[i, t] * dd
            r, re = a[t] * r, a[t] * (re + r * fade[t])
        out[8][i] = re + U * r
    channels = (D // G + 8) * U                              # roundings of the sums over a group's channels
    out[3], out[4] = join(out[3] + channels * dbm), join(out[4] + channels * dcm)
    return (ye, fe), tuple(out)


GRADS = ("dx", "ddt", "dA", "db", "dc", "dskip", "dgate", "ddt_bias", "d initial")
SCAN_IN = ("x", "dt", "A", "b", "c", "skip", "gate", "dt_bias")


def check_scan(a, dtype, lengths=None, softplus=True, backward=True, label=""):
    print(f"[scan] {dtype} x{tuple(a['x'].shape)} b{tuple(a['b'].shape)} lengths={lengths} softplus={softplus} "
          f"gate={a['gate'] is not None} initial={a['initial_state'] is not None} {label}", flush=True)
    h = {k: _n(v) for k, v in a.items()}
    kw = dict(skip=a["skip"], gate=a["gate"], dt_bias=a["dt_bias"], softplus=softplus, initial_state=a["initial_state"],
              lengths=_lengths(lengths))
    ho = dict(softplus=softplus, initial_state=h["initial_state"], lengths=lengths)
    want = ref.ssm_scan(*(h[k] for k in SCAN_IN), **ho)
    (ye, fe), errs = scan_bounds(h, lengths, softplus)
    y, final = pn.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"], **kw)
    _close(y, want[0], _bound(dtype, want[0], ye), "y")
    _close(final, want[1], 1.01 * fe + U * np.abs(want[1]), "final state")
    if not backward:
        return
    got = pn.ssm_scan_backward(a["dy"], a["x"], a["dt"], a["A"], a["b"], a["c"], d_final_state=a["d_final_state"], **kw)
    want = ref.ssm_scan_backward(h["dy"], *(h[k] for k in SCAN_IN), d_final_state=h["d_final_state"], **ho)
    absent = dict(dskip="skip", dgate="gate", ddt_bias="dt_bias")
    for x, w, e, name in zip(got, want, errs, GRADS):
        if (name in absent and a[absent[name]] is None) or (name == "d initial" and a["initial_state"] is None):
            assert x is None, name
            continue
        stored = dtype if name in ("dx", "ddt", "db", "dc", "dgate") else "f32"
        _close(x, w, _bound(stored, w, e), name)


SCAN = [  # B, T, D, N, G
    (1, 1, 1, 1, 1), (2, 1, 64, 16, 1), (1, 7, 5, 3, 1), (2, 8, 65, 4, 1), (1, 9, 66, 5, 2), (2, 17, 130, 8, 2), (1, 40, 63, 12, 1),
    (3, 33, 128, 16, 4), (1, 100, 70, 16, 1), (1, 20, 30, 17, 1), (2, 24, 65, 32, 1), (1, 19, 12, 100, 3), (1, 33, 20, 128, 1),
    (2, 200, 64, 16, 1)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SCAN, ids=["x".join(map(str, s)) for s in SCAN])
def test_scan_shapes(dtype, shape):
    check_scan(scan_inputs(dtype, *shape), dtype)
    check_scan(scan_inputs(dtype, *shape, initial=False, gate=False, seed=1), dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [4, 8, 16, 40])
def test_scan_lengths(dtype, N):
    """Sequences that end at every place of a tile and of a segment; padding is never read, and its rows are 0."""
    B, T, D = 7, 200, 40
    a = scan_inputs(dtype, B, T, D, N, 2)
    n, given = [0, 1, 8, 63, 64, 137, 200], [-3, 1, 8, 63, 64, 137, 100000]
    check_scan(a, dtype, lengths=n)
    dirty = {k: None if v is None else v.clone() for k, v in a.items()}
    for b, m in enumerate(n):
        for k in ("x", "dt", "b", "c", "gate", "dy"):
            dirty[k][b, m:] = float("nan")
    kw = dict(skip=a["skip"], dt_bias=a["dt_bias"], initial_state=a["initial_state"])
    for f, first in ((pn.ssm_scan, ()), (pn.ssm_scan_backward, ("dy",))):
        more = dict(d_final_state=a["d_final_state"]) if first else {}
        got = [f(*[v[k] for k in first + ("x", "dt", "A", "b", "c")], gate=v["gate"], lengths=_lengths(m), **kw, **more)
               for v, m in ((dirty, given), (a, n))]
        for x, y in zip(*got):
            assert torch.equal(x, y) and bool(torch.isfinite(x).all())
    y, final = pn.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"], gate=a["gate"], lengths=_lengths(given), **kw)
    assert torch.equal(final[0], a["initial_state"][0])
    for b, m in enumerate(n):
        assert not y[b, m:].any()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_scan_options(dtype):
    for drop in (("skip",), ("dt_bias",), ("skip", "dt_bias", "gate"), ("d_final_state",)):
        a = scan_inputs(dtype, 2, 37, 24, 16, 1)
        a.update((k, None) for k in drop)
        check_scan(a, dtype)
    a = scan_inputs(dtype, 2, 37, 24, 16, 1)
    a["dt"] = a["dt"].abs() * 0.2
    a["dt_bias"] = a["dt_bias"].abs() * 0.1
    check_scan(a, dtype, softplus=False)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("step, rate", [(1e-4, 0.01), (0.5, 30.0), (20.0, 3.0), (0.05, -0.5), (0.1, 0.0)])
def test_scan_steps_and_decays(dtype, step, rate):
    """Long memories, decays that underflow, steps past the bend of the softplus, growth, and no decay at all."""
    a = scan_inputs(dtype, 1, 100, 64, 16, 1, step=min(step, 5.0))
    if step > 5.0:
        a["dt_bias"] = torch.full_like(a["dt_bias"], step)
    a["A"] = torch.full_like(a["A"], -rate)
    check_scan(a, dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_scan_strides(dtype):
    g = torch.Generator().manual_seed(3)
    B, T, D, N, G = 2, 50, 36, 16, 2
    a = scan_inputs(dtype, B, T, D, N, G)
    packed = _rand(g, (B, T, 3 * D + 2 * G * N + 1), dtype)
    a["x"], a["gate"] = packed[..., 1:1 + D], packed[..., 1 + D:1 + 2 * D]
    a["dt"] = packed[..., 1 + 2 * D:1 + 3 * D]
    a["b"] = packed[..., 1 + 3 * D:1 + 3 * D + G * N].unflatten(-1, (G, N))
    a["c"] = packed[..., 1 + 3 * D + G * N:].unflatten(-1, (G, N))
    a["dy"] = _rand(g, (T, B, D), dtype).transpose(0, 1)
    check_scan(a, dtype, label="packed")
    a["b"] = a["b"][:, :, :1].expand(B, T, G, N)             # one group shared by stride 0
    a["c"] = a["c"][:1].expand(B, T, G, N)
    check_scan(a, dtype, label="broadcast")


@pytest.mark.parametrize("dtype", list(TYPES))
def test_scan_segments(dtype):
    """A long text in many segments, from and to a state: as the oracle, and as one sequence cut in two calls."""
    a = scan_inputs(dtype, 1, 1000, 64, 16, 1, step=0.01)
    check_scan(a, dtype)
    kw = dict(skip=a["skip"], dt_bias=a["dt_bias"])
    names = ("x", "dt", "b", "c", "gate")
    cut = lambda s: {k: a[k][:, s] for k in names}  # noqa: E731
    first, last = cut(slice(0, 333)), cut(slice(333, None))
    y0, h = pn.ssm_scan(first["x"], first["dt"], a["A"], first["b"], first["c"], gate=first["gate"],
                        initial_state=a["initial_state"], **kw)
    y1, h1 = pn.ssm_scan(last["x"], last["dt"], a["A"], last["b"], last["c"], gate=last["gate"], initial_state=h, **kw)
    y, final = pn.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"], gate=a["gate"], initial_state=a["initial_state"], **kw)
    host = {k: _n(v) for k, v in a.items()}
    (ye, fe), _ = scan_bounds(host, None)
    _close(torch.cat((y0, y1), 1), _np(y), 2 * (_bound(dtype, _np(y), ye)), "two calls")
    _close(h1, _np(final), 2.1 * fe, "state of two calls")


@pytest.mark.parametrize("T", list(range(1, 34)) + [63, 64, 65, 81, 95, 96, 97, 127, 128, 129, 143, 161, 257, 513, 1100])
def test_scan_lengths_of_one_call(T):
    """Every length of the first tiles, and those at which segments begin."""
    check_scan(scan_inputs("bf16", 1, T, 40, 16, 1, seed=T), "bf16")


def test_one_token_with_any_token_stride():
    """The stride of a single token is never used."""
    for st in (1 << 20, 1 << 27, 1 << 33):
        a, c, n = scan_inputs("bf16", 2, 1, 40, 16, 2), conv_inputs("bf16", 2, 1, 40, 4, True), norm_inputs("bf16", "f32", (2, 1), 40)
        far = lambda t: t.as_strided(t.shape, (t.stride(0), st, *t.stride()[2:]))  # noqa: E731
        check_scan({k: far(v) if k in ("x", "dt", "b", "c", "gate", "dy") else v for k, v in a.items()}, "bf16")
        check_conv({k: far(v) if k in ("x", "dy") else v for k, v in c.items()}, "bf16")
        check_norm({k: far(v) if v.dim() == 3 else v for k, v in n.items()}, "bf16", "f32")


def test_scan_without_tokens():
    a = scan_inputs("bf16", 2, 0, 24, 16, 1)
    y, final = pn.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"], initial_state=a["initial_state"])
    assert y.shape == (2, 0, 24) and torch.equal(final, a["initial_state"])
    assert not pn.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"])[1].any()
    for B in (2, 0):
        v = {k: a[k][:B] for k in ("dy", "x", "dt", "b", "c", "gate", "initial_state", "d_final_state")}
        back = pn.ssm_scan_backward(v["dy"], v["x"], v["dt"], a["A"], v["b"], v["c"], skip=a["skip"], gate=v["gate"],
                                    dt_bias=a["dt_bias"], initial_state=v["initial_state"], d_final_state=v["d_final_state"])
        assert torch.equal(back[8], v["d_final_state"])
        assert not any(back[i].any() for i in (2, 5, 7))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("D, N, G", [(24, 16, 1), (33, 5, 3), (10, 1, 1), (8, 64, 2), (6, 100, 1), (4, 127, 1), (4, 128, 1)])
def test_scan_steps_against_the_oracle(dtype, D, N, G):
    """Single tokens on a pool, idle rows between.  Every step starts from the state as it is, so the bounds are those of
    one token."""
    B, T = 5, 4
    a = scan_inputs(dtype, B, T, D, N, G)
    slots = torch.tensor([6, -1, 0, 2, 7], dtype=torch.int32, device=DEV)
    pool = torch.full((7, D, N), 7.0, device=DEV)
    live = [0, 2, 3]
    at = [6, 0, 2]
    pool[at] = a["initial_state"][live]
    kw = dict(skip=a["skip"], dt_bias=a["dt_bias"])
    for t in range(T):
        before = _np(pool)
        y = pn.ssm_step(a["x"][:, t], a["dt"][:, t], a["A"], a["b"][:, t], a["c"][:, t], pool, gate=a["gate"][:, t], slots=slots, **kw)
        h = {k: (_n(a[k]) if k in ("A", "skip", "dt_bias") else _n(a[k][:, t:t + 1])[live]) for k in
             ("x", "dt", "A", "b", "c", "skip", "gate", "dt_bias", "dy")}
        h.update(initial_state=before[at], d_final_state=None)
        want = ref.ssm_scan(*(h[k] for k in SCAN_IN), initial_state=before[at])
        (ye, fe), _ = scan_bounds(h, None)
        _close(y[live], want[0][:, 0], _bound(dtype, want[0], ye)[:, 0], "y")
        _close(pool[at], want[1], 1.01 * fe + U * np.abs(want[1]), "state")
        assert not y[[1, 4]].any() and bool((pool[[1, 3, 4, 5]] == 7.0).all())


# ---------------------------------------------------------------- norms around a block


def norm_inputs(dtype, rdtype, lead, D, seed=0):
    g = torch.Generator().manual_seed(seed)
    a = {k: _rand(g, (*lead, D), dtype) for k in ("x", "gate", "dy")}
    a["residual"], a["ds"] = _rand(g, (*lead, D), rdtype, 2.0), _rand(g, (*lead, D), rdtype, 0.5)
    for k in ("weight", "post_weight", "scale"):
        a[k] = 1.0 + _rand(g, (D,), "f32", 0.3)
    return a


def check_norm(a, dtype, rdtype, eps=1e-5, backward=True):
    print(f"[norm] {dtype} {rdtype} x{tuple(a['x'].shape)} " + " ".join(k for k in ("residual", "gate", "post_weight", "scale", "weight")
                                                                       if a[k] is not None), flush=True)
    h = {k: _n(v) for k, v in a.items()}
    kw = {k: a[k] for k in ("gate", "post_weight", "scale")}
    hk = {k: h[k] for k in ("gate", "post_weight", "scale")}
    y, s = pn.block_norm(a["x"], a["weight"], residual=a["residual"], eps=eps, **kw)
    wy, ws = ref.block_norm(h["x"], h["weight"], h["residual"], eps=eps, **hk)
    zmax = 0.0 if a["gate"] is None else float(np.abs(h["gate"]).max())
    # u and the mean of its squares: silu's error, and 40 roundings of sums in lanes, waves and between
    k = (2 * zmax + 48) * U
    p = ws - (0.0 if h["residual"] is None else h["residual"])
    se = 2 * k * np.abs(p) + 2 * U * (np.abs(ws) + np.abs(p))
    _close(s, ws, _bound(rdtype, ws, se), "s")
    if a["weight"] is None:
        assert y is None
    else:
        far = np.sqrt((se * se).sum(-1, keepdims=True) / np.maximum((ws * ws).sum(-1, keepdims=True), 1e-300))
        rs = 1.0 / np.sqrt((ws * ws).mean(-1, keepdims=True) + eps)
        _close(y, wy, _bound(dtype, wy, np.abs(h["weight"]) * rs * se + np.abs(wy) * (far + 40 * U)), "y")
    if not backward:
        return
    got = pn.block_norm_backward(a["dy"] if a["weight"] is not None else None, a["ds"], a["x"], a["weight"],
                                 residual=a["residual"], eps=eps, **kw)
    want, mag = ref.block_norm_backward(h["dy"], h["ds"], h["x"], h["weight"], h["residual"], eps=eps, **hk)
    # the roundings of s are relative to its terms, |residual| + |p|, and so is what they do to its norm
    terms = np.abs(p) + (0.0 if h["residual"] is None else np.abs(h["residual"]))
    far = np.sqrt((terms ** 2).sum(-1) / np.maximum((ws ** 2).sum(-1), 1e-300)).max()
    n = (8 * zmax + 160) * (1.0 + far) * U
    for x, w, m, name in zip(got, want, mag, ("dx", "dweight", "dresidual", "dgate", "dpost_weight", "dscale")):
        if w is None:
            assert x is None, name
            continue
        stored = {"dresidual": rdtype, "dx": dtype, "dgate": dtype}.get(name, "f32")
        e = n * m
        if name == "dgate":                                  # the slope's error is relative to its terms, not to itself
            z = h["gate"]
            pr = ref.logistic(z)
            slope = np.abs(pr * (1 + z * (1 - pr)))
            e = m * n + m / np.maximum(slope, 1e-300) * pr * (1 + np.abs(z)) * (2 * np.abs(z) + 10) * U
        _close(x, w, _bound(stored, w, e), name)


PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")]
NORM_D = [1, 2, 7, 64, 66, 130, 512, 1000, 1024, 2048, 2050, 4096, 4104, 8192]


@pytest.mark.parametrize("dtype, rdtype", PAIRS)
@pytest.mark.parametrize("D", NORM_D)
def test_norm_widths(dtype, rdtype, D):
    check_norm(norm_inputs(dtype, rdtype, (2, 3), D), dtype, rdtype)


@pytest.mark.parametrize("dtype, rdtype", PAIRS)
@pytest.mark.parametrize("D", [40, 1024, 2048])
def test_norm_many_rows(dtype, rdtype, D):
    """Past the number of rows from which a wave takes a row."""
    check_norm(norm_inputs(dtype, rdtype, (3, 700), D), dtype, rdtype)


@pytest.mark.parametrize("dtype, rdtype", [("f32", "f32"), ("bf16", "f32")])
def test_norm_widest(dtype, rdtype):
    for D in (2049, 2560, 2561, 2562, 4097, 5000, 8191):
        check_norm(norm_inputs(dtype, rdtype, (1, 3), D), dtype, rdtype)


@pytest.mark.parametrize("dtype, rdtype", PAIRS)
@pytest.mark.parametrize("drop", [("gate",), ("post_weight",), ("scale",), ("weight",), ("residual",), ("ds",),
                                  ("gate", "post_weight", "scale"), ("post_weight", "scale"), ("gate", "post_weight", "scale", "residual"),
                                  ("weight", "post_weight", "scale"), ("weight", "scale")])
def test_norm_options(dtype, rdtype, drop):
    a = norm_inputs(dtype, rdtype, (2, 9), 72)
    a.update((k, None) for k in drop)
    if "residual" in drop:
        if dtype != rdtype:
            return                                           # without a residual s has the tokens' type
        a["ds"] = a["ds"].to(TYPES[dtype])
    check_norm(a, dtype, rdtype)


@pytest.mark.parametrize("dtype, rdtype", PAIRS)
def test_norm_strides_and_single_tokens(dtype, rdtype):
    g = torch.Generator().manual_seed(4)
    a = norm_inputs(dtype, rdtype, (3, 5), 48)
    packed = _rand(g, (3, 5, 2 * 48 + 1), dtype)
    a["x"], a["gate"] = packed[..., 1:49], packed[..., 49:]
    a["residual"] = _rand(g, (5, 3, 48), rdtype).transpose(0, 1)
    a["ds"] = a["ds"][:, :1].expand(3, 5, 48)
    check_norm(a, dtype, rdtype)
    check_norm({k: v[:, 0] if v.dim() == 3 else v for k, v in a.items()}, dtype, rdtype)


def test_norm_of_wide_rows_is_captured():
    """Rows whose weights take more LDS than a launch has by itself."""
    a = norm_inputs("bf16", "bf16", (1, 5), 8192)
    kw = {k: a[k] for k in ("gate", "post_weight", "scale")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pn.block_norm_backward(a["dy"], a["ds"], a["x"], a["weight"], residual=a["residual"], **kw)
    for i in range(3):
        a["dy"].mul_(1.5)
        graph.replay()
        want = pn.block_norm_backward(a["dy"], a["ds"], a["x"], a["weight"], residual=a["residual"], **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)), i


def test_norm_without_tokens():
    a = norm_inputs("bf16", "f32", (2, 0), 64)
    kw = {k: a[k] for k in ("gate", "post_weight", "scale")}
    y, s = pn.block_norm(a["x"], a["weight"], residual=a["residual"], **kw)
    assert y.shape == (2, 0, 64) and s.dtype is torch.float32
    back = pn.block_norm_backward(a["dy"], a["ds"], a["x"], a["weight"], residual=a["residual"], **kw)
    assert not any(back[i].any() for i in (1, 4, 5))


def test_norm_rows_of_zeros_and_far_values():
    for dtype in TYPES:
        a = norm_inputs(dtype, dtype, (1, 4), 64)
        for k in ("x", "residual"):
            a[k][0, 1] = 0.0
        a["x"][0, 2] = float("nan")
        y, s = pn.block_norm(a["x"], a["weight"], residual=a["residual"], post_weight=a["post_weight"])
        assert not y[0, 1].any() and not s[0, 1].any()
        assert bool(torch.isnan(y[0, 2]).all()) and bool(torch.isfinite(y[0, [0, 3]]).all())
        check_norm({k: v if v.dim() == 1 else v[:, [0, 3]] for k, v in a.items()}, dtype, dtype)


# ---------------------------------------------------------------- all of them


def _calls():
    """(name, inputs, f(inputs) -> outputs) of every entry, the pools of the steps among the outputs."""
    c, s, n = conv_inputs("bf16", 2, 150, 64, 4, True), scan_inputs("bf16", 2, 150, 64, 16, 1), norm_inputs("bf16", "f32", (2, 150), 64)
    kc = ("bias", "initial_state")
    ks = ("skip", "gate", "dt_bias", "initial_state")
    kn = ("gate", "post_weight", "scale")
    pick = lambda a, k: {x: a[x] for x in k}  # noqa: E731
    one = {k: v[:, 0] if k in ("x", "dt", "b", "c", "gate", "dy") else v for k, v in s.items()}
    return [
        ("conv", c, lambda a: pn.short_conv(a["x"], a["weight"], **pick(a, kc))),
        ("conv gradients", c, lambda a: pn.short_conv_backward(a["dy"], a["x"], a["weight"], d_final_state=a["d_final_state"], **pick(a, kc))),
        ("conv step", dict(c, x=c["x"][:, 0]), lambda a: (pn.short_conv_step(a["x"], a["weight"], a["initial_state"], bias=a["bias"]),
                                                         a["initial_state"])),
        ("scan", s, lambda a: pn.ssm_scan(*(a[k] for k in ("x", "dt", "A", "b", "c")), **pick(a, ks))),
        ("scan gradients", s, lambda a: pn.ssm_scan_backward(*(a[k] for k in ("dy", "x", "dt", "A", "b", "c")),
                                                             d_final_state=a["d_final_state"], **pick(a, ks))),
        ("scan step", one, lambda a: (pn.ssm_step(*(a[k] for k in ("x", "dt", "A", "b", "c")), a["initial_state"], **pick(a, ks[:3])),
                                      a["initial_state"])),
        ("norm", n, lambda a: pn.block_norm(a["x"], a["weight"], residual=a["residual"], **pick(a, kn))),
        ("norm gradients", n, lambda a: pn.block_norm_backward(a["dy"], a["ds"], a["x"], a["weight"], residual=a["residual"],
                                                                **pick(a, kn))),
    ]


def _copy(a):
    return {k: None if v is None else v.clone() for k, v in a.items()}


@pytest.mark.parametrize("which", range(8))
def test_same_bits_on_every_run_and_stream(which):
    name, a, f = _calls()[which]
    want = f(_copy(a))
    other = torch.cuda.Stream()
    for _ in range(3):
        mine = _copy(a)
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            got = f(mine)
        torch.cuda.current_stream().wait_stream(other)
        for x, y in zip(got, want):
            assert torch.equal(x, y), name


@pytest.mark.parametrize("which", range(8))
def test_captured_and_replayed(which):
    """A captured call, replayed on changed inputs with eager work between, gives what an eager call gives."""
    name, a, f = _calls()[which]
    held = _copy(a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        f(_copy(a))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = f(held)
    for i in range(4):
        fresh = {k: None if v is None else v * (1.0 + 0.25 * i) for k, v in a.items()}
        for k, v in fresh.items():
            if v is not None:
                held[k].copy_(v)
        graph.replay()
        want = f(_copy(fresh))
        torch.cuda.synchronize()
        for x, y in zip(out, want):
            assert torch.equal(x, y), (name, i)
