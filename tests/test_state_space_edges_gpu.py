"""State-space operators on the GPU where sizes, splits and values are extreme.

Tolerances are those of test_state_space_gpu.py unless a test derives its own.
"""

import numpy as np
import pytest
import torch

import newton_evaluation_nonlinear_amd as pn
from newton_evaluation_nonlinear_amd import state_space as ss
from oracle import state_space as ref
from test_sequence_gpu import DEV, TINY, TYPES, _np
from test_state_space_gpu import PAIRS, U, check_norm, check_scan, conv_inputs, norm_inputs, scan_inputs

pytestmark = pytest.mark.gpu


def scan_bytes(B, T, D, N, G, wide, segments):
    """Workspace of the scan's gradients with `wide` channel blocks a workgroup and `segments` of the time axis."""
    states, blocks = (4 if N <= 4 else 8 if N <= 8 else 16), -(-N // 16)
    per_group = -(-(-(-(D // G) // 32)) // wide) * wide
    tiles, chans = -(-T // 8), G * per_group
    rows = B * chans
    state = rows * blocks * states * 32
    parts = [tiles * state, tiles * rows * 32, chans // wide * B * T * 2 * blocks * states, B * segments * D * N,
             B * segments * blocks * 2 * D]
    if segments > 1:
        parts += [segments * state, segments * rows * 32, segments * state]
    return 4 * sum(-(-n // 64) * 64 for n in parts)


def scan_splits(B, T, D, N, G):
    """(channel blocks of a workgroup, segments) of the scan's gradients: those that its workspace has room for."""
    n = pn.lib().pn_ssm_scan_workspace_bytes(ss._SSM(0, B, T, D, N, G, 1, *[0] * 44), 1)
    return [(wide, k) for wide in (1, 2, 4) for k in range(1, min(T, 300) // 8 + 2) if n == scan_bytes(B, T, D, N, G, wide, k)]


def norm_groups(rows, D):
    """Workgroups of the norm's gradients, from the workspace that holds three rows of each."""
    return pn.lib().pn_block_norm_workspace_bytes(ss._NORM(0, 0, 1, rows, D, 1e-5, 1, 1, 1, *[0] * 31)) / (12 * D)


# ---------------------------------------------------------------- splits


# B, T, D, N, G, channel blocks of a workgroup of the gradients, segments, lengths
WIDE = [(1, 20, 128, 16, 1, 4, 1, None),                 # one share of db and dc
        (3, 23, 256, 12, 1, 4, 1, [23, 0, 9]),           # two
        (2, 96, 128, 3, 1, 4, 12, [96, 37]),             # in segments
        (1, 40, 512, 8, 1, 4, 5, [33]),
        (2, 22, 256, 16, 2, 4, 1, [22, 17]),             # two groups
        (2, 50, 480, 16, 1, 4, 4, [50, 8]),              # 15 blocks and one without a channel
        (1, 17, 257, 16, 1, 2, 1, None),                 # 9 blocks, the last of one channel, and one without
        (2, 29, 288, 5, 1, 2, 2, [29, 24]),
        (1, 21, 1026, 4, 2, 2, 1, None),                 # 17 and one without, twice
        (1, 18, 64, 16, 1, 2, 1, None),
        (8, 90, 2048, 3, 1, 4, 1, [90, 89, 65, 64, 63, 8, 1, 0]),   # sums over more than 64 tokens of a segment
        (64, 75, 6, 128, 1, 1, 1, None)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("case", WIDE, ids=["x".join(map(str, c[:5])) for c in WIDE])
def test_scan_gradients_of_wide_groups(dtype, case):
    """Workgroups of several channel blocks, that add their shares of db and dc in LDS; and long single segments."""
    *sizes, _, _, lengths = case
    check_scan(scan_inputs(dtype, *sizes), dtype, lengths=lengths)


ROWS = [(40, 6200), (512, 6200), (514, 3100), (2048, 1550), (2050, 1100), (2559, 1100), (2560, 1100), (4096, 601), (4097, 601),
        (4104, 601), (8191, 601), (8192, 601)]


@pytest.mark.parametrize("dtype, rdtype", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("D, rows", ROWS)
def test_norm_gradients_of_several_rows_a_workgroup(dtype, rdtype, D, rows):
    """Three rows for each workgroup of the gradients, and fewer for the last."""
    check_norm(norm_inputs(dtype, rdtype, (1, rows), D), dtype, rdtype)


# ---------------------------------------------------------------- masked values


def _same(got, want):
    for x, y in zip(got, want):
        assert (x is None) == (y is None)
        if x is not None:
            assert bool(torch.isfinite(y).all()) and torch.equal(x, y)


@pytest.mark.parametrize("dtype, rdtype", PAIRS)
@pytest.mark.parametrize("D", [7, 64, 2050, 4104, 8192])
@pytest.mark.parametrize("post", [True, False])
def test_norm_gates_of_the_lowest_value(dtype, rdtype, D, post, monkeypatch):
    """A gate of the type's lowest value lets through what one of -200 does: v sigmoid(v) and its slope are 0 in float32
    there (200 e^-200 is 1e-85), so outputs and gradients are the same bits, and those of -200 are the oracle's.  To the
    tolerance comes half the smallest subnormal of float32 and bfloat16, below which a result is rounded to 0."""
    a = norm_inputs(dtype, rdtype, (2, 4), D)
    a["x"], a["dy"] = a["x"] * 4, a["dy"] * 4
    if not post:
        a["post_weight"] = None
    off = torch.zeros(2, 4, D, dtype=torch.bool, device=DEV)
    off[0, 1], off[1, 2, ::3] = True, True
    results = []
    for value in (torch.finfo(TYPES[dtype]).min, -200.0):
        a["gate"] = torch.where(off, value, a["gate"].float()).to(TYPES[dtype])
        kw = {k: a[k] for k in ("residual", "gate", "post_weight", "scale")}
        results.append(pn.block_norm(a["x"], a["weight"], **kw) + pn.block_norm_backward(a["dy"], a["ds"], a["x"], a["weight"], **kw))
    _same(*results)
    for t, bits in (("f32", 150), ("bf16", 134)):
        monkeypatch.setitem(TINY, t, 2.0 ** -bits)
    check_norm(a, dtype, rdtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [8, 16, 40])
def test_scan_gates_of_the_lowest_value(dtype, N):
    a = scan_inputs(dtype, 2, 70, 40, N, 1)
    off = torch.zeros(2, 70, 40, dtype=torch.bool, device=DEV)
    off[0, 9], off[1, :, ::3] = True, True
    results = []
    for value in (torch.finfo(TYPES[dtype]).min, -200.0):
        z = torch.where(off, value, a["gate"].float()).to(TYPES[dtype])
        kw = dict(skip=a["skip"], dt_bias=a["dt_bias"])
        args = (a["x"], a["dt"], a["A"], a["b"], a["c"])
        pool = a["initial_state"].clone()
        step = pn.ssm_step(a["x"][:, 9], a["dt"][:, 9], a["A"], a["b"][:, 9], a["c"][:, 9], pool, gate=z[:, 9], **kw)
        kw.update(gate=z, initial_state=a["initial_state"])
        results.append(pn.ssm_scan(*args, **kw) + pn.ssm_scan_backward(a["dy"], *args, d_final_state=a["d_final_state"], **kw) + (step, pool))
    _same(*results)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [8, 16, 40])
@pytest.mark.parametrize("closed", ["lowest", "infinite"])
def test_scan_steps_closed_by_a_mask(dtype, N, closed):
    """dt of the type's lowest value or minus infinity is a step of 0, as is that of -200: the state is kept."""
    a = scan_inputs(dtype, 2, 70, 40, N, 1)
    off = torch.zeros(2, 70, 40, dtype=torch.bool, device=DEV)
    off[0, 9], off[1, :, ::3], off[1, 30:50] = True, True, True
    results = []
    for value in (torch.finfo(TYPES[dtype]).min if closed == "lowest" else -float("inf"), -200.0):
        dt = torch.where(off, value, a["dt"].float()).to(TYPES[dtype])
        kw = dict(skip=a["skip"], dt_bias=a["dt_bias"])
        pool = a["initial_state"].clone()
        step = pn.ssm_step(a["x"][:, 9], dt[:, 9], a["A"], a["b"][:, 9], a["c"][:, 9], pool, gate=a["gate"][:, 9], **kw)
        assert torch.equal(pool[0], a["initial_state"][0])
        args = (a["x"], dt, a["A"], a["b"], a["c"])
        kw.update(gate=a["gate"], initial_state=a["initial_state"])
        results.append(pn.ssm_scan(*args, **kw) + pn.ssm_scan_backward(a["dy"], *args, d_final_state=a["d_final_state"], **kw) + (step, pool))
    _same(*results)


@pytest.mark.parametrize("dtype", list(TYPES))
def test_conv_biases_of_the_lowest_value(dtype):
    """Channels that their bias closes, as one of -1000 does."""
    a = conv_inputs(dtype, 2, 70, 40, 4, True)
    results = []
    for value in (torch.finfo(torch.float32).min, -1000.0):
        bias = a["bias"].clone()
        bias[::3] = value
        kw = dict(bias=bias, initial_state=a["initial_state"])
        pool = a["initial_state"].clone()
        results.append(pn.short_conv(a["x"], a["weight"], **kw)
                       + pn.short_conv_backward(a["dy"], a["x"], a["weight"], d_final_state=a["d_final_state"], **kw)
                       + (pn.short_conv_step(a["x"][:, 0], a["weight"], pool, bias=bias), pool))
    _same(*results)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("N", [3, 8, 16, 40])
@pytest.mark.parametrize("T", [13, 200])
def test_scan_decays_of_the_lowest_value(dtype, N, T):
    """A of float32's lowest value forgets everything at every step above 1e-28, as -1e30 does: the same bits, those of -1e30
    the oracle's, in sequences that end inside a tile too.  A step of 0 (softplus of -200) keeps the state."""
    a = scan_inputs(dtype, 3, T, 40, N, 1)
    a["A"] = a["A"].clone()
    lengths = [T, T - 3, 1]
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    closed = a["dt"].clone()
    closed[0, 5:9] = -200.0
    results = []
    for value in (torch.finfo(torch.float32).min, -1e30):
        a["A"][:, ::2] = value
        kw = dict(skip=a["skip"], gate=a["gate"], dt_bias=a["dt_bias"], initial_state=a["initial_state"], lengths=n)
        rest = (a["A"], a["b"], a["c"])
        results.append(pn.ssm_scan(a["x"], closed, *rest, **kw) + pn.ssm_scan(a["x"], a["dt"], *rest, **kw)
                       + pn.ssm_scan_backward(a["dy"], a["x"], a["dt"], *rest, d_final_state=a["d_final_state"], **kw))
    _same(*results)
    check_scan(a, dtype, lengths=lengths)


# ---------------------------------------------------------------- long sums


@pytest.mark.parametrize("B, N", [(2048, 1), (1024, 20), (256, 128)])
def test_scan_sums_over_a_long_segment(B, N):
    """Sums over 16384 tokens of one segment, of terms of one sign and (after the first few) one size, which a single float32
    sum would leave by 2e-5 and more of itself.

    Every sequence is the same, so the sums are B times the oracle's of one.  With A = -1 and steps of about 2 a decay,
    e^-2 = 0.13, is off by at most 9 U of itself (the step's rounding and two of the exponent, times 2, and two more), a state
    and its gradient by (0.13 * 10 + 0.87 * 3 + 1) U / 0.87 < 6 U, a kept state by 16, the terms of dA by 25 and those of
    dskip by 1.  The terms of ddt_bias are sums over N states: 30 + 2 N, for what each term and the sums in lanes and
    waves take.  64 terms are added in float32, which is 64 U at most; the rest of the sum is float64, rounded twice."""
    T, v = 16384, 0.7234
    same = lambda *s: torch.full(s, v, device=DEV).expand(B, *s[1:])  # noqa: E731
    x, b, dt = same(1, T, 1), same(1, T, 1, N), same(1, T, 1) + 0.6
    A, skip, bias = -torch.ones(1, N, device=DEV), torch.full((1,), v, device=DEV), torch.full((1,), v, device=DEV)
    assert scan_splits(B, T, 1, N, 1) == [(1, 1)]
    got = pn.ssm_scan_backward(x, x, dt, A, b, b, skip=skip, dt_bias=bias, softplus=False)
    one = [_np(t[:1]) for t in (x, x, dt)] + [_np(A), _np(b[:1]), _np(b[:1]), _np(skip), None, _np(bias)]
    want, mag = (ref.ssm_scan_backward(*one, softplus=False, bound=bound) for bound in (False, True))
    for i, n in ((2, 25), (5, 1), (7, 30 + 2 * N)):
        assert (np.abs(_np(got[i]) / B - want[i]) <= (n + 66) * U * mag[i]).all(), (i, _np(got[i]) / B, want[i])


@pytest.mark.parametrize("D, rows", [(4, (1 << 23) + 5), (600, 2000000)])
def test_norm_sums_over_many_rows(D, rows):
    """Sums over many equal rows, which a single float32 sum of a workgroup's (2731 of 4 channels, 1303 of 600) would leave by
    more than the bound.

    A term is off by less than 40 U of itself (the mean of D squares in lanes and waves: 12 roundings of its terms, so 6 of
    its root, twice; root, reciprocal, products, and the mean in t, of the size of its terms).  At most 128 terms are added
    in float32, the rest in float64, rounded twice; the sums are `rows` times the oracle's of one row."""
    g = torch.Generator().manual_seed(3)
    row = (torch.rand(1, 1, D, generator=g) + 0.5).to(DEV)
    x = row.expand(1, rows, D)
    w = torch.ones(D, device=DEV)
    got = pn.block_norm_backward(x, None, x, w, post_weight=w, scale=w)
    want, mag = ref.block_norm_backward(_np(row), None, _np(row), _np(w), None, None, _np(w), _np(w))
    for i in (1, 4, 5):
        assert (np.abs(_np(got[i]) / rows - want[i]) <= (40 + 130) * U * mag[i]).all(), i
    assert norm_groups(rows, D) >= rows // 128


# ---------------------------------------------------------------- far rows


def _far(dtype, D, by, g):
    """[1, 3, D] of elements of `by` times the size at which their squares sum to float32's largest value."""
    size = by * float(np.sqrt(np.finfo(np.float32).max / D))
    return (torch.where(torch.rand(1, 3, D, generator=g) < 0.5, -size, size)).to(DEV).to(TYPES[dtype])


@pytest.mark.parametrize("dtype, rdtype", [p for p in PAIRS if p[0] != "f16"])
@pytest.mark.parametrize("D", [1, 7, 64, 2048, 2050, 8192])
def test_norm_rows_on_both_sides_of_float32(dtype, rdtype, D):
    """Rows whose squares just fit float32 are normed like others; past it they come out as 0 and pass no gradient, also
    where the sums of the gradient's products do not fit either.  (bfloat16 is within 2^-8 of the sizes given.)"""
    g = torch.Generator().manual_seed(D)
    a = norm_inputs(dtype, rdtype, (1, 3), D)
    a["gate"] = None
    plain = dict(a, post_weight=None)
    check_norm(dict(plain, residual=_far(rdtype, D, 0.99, g)), dtype, rdtype)
    check_norm(dict(a, x=_far(dtype, D, 0.99, g)), dtype, rdtype)
    for dy in (a["dy"], torch.full_like(a["dy"], 1e25)):
        far = dict(plain, residual=_far(rdtype, D, 1.01, g))         # past it in s
        y, s = pn.block_norm(far["x"], far["weight"], residual=far["residual"], scale=far["scale"])
        dx, dw, dr, _, _, dsc = pn.block_norm_backward(dy, far["ds"], far["x"], far["weight"], residual=far["residual"], scale=far["scale"])
        assert not y.any() and not dw.any() and bool(torch.isfinite(s).all()) and torch.equal(dr, far["ds"])
        assert torch.equal(dx, (far["ds"].float() * far["scale"]).to(dx.dtype))
        want = (far["ds"].double() * far["x"].double()).sum((0, 1))
        assert bool(((dsc.double() - want).abs() <= 8 * U * (far["ds"].double() * far["x"].double()).abs().sum((0, 1))).all())
    x = _far(dtype, D, 1.01, g)                                      # past it in u: with a large gradient of s
    ds = torch.full_like(a["ds"], 1e25)
    kw = dict(residual=a["residual"], post_weight=a["post_weight"], scale=a["scale"])
    y, s = pn.block_norm(x, a["weight"], **kw)
    assert torch.equal(s, a["residual"]) and bool(torch.isfinite(y).all())
    dx, dw, dr, _, dpw, dsc = pn.block_norm_backward(a["dy"], ds, x, a["weight"], **kw)
    assert not dx.any() and not dpw.any() and not dsc.any() and torch.equal(dr, ds)


# ---------------------------------------------------------------- past 2^32 elements


def test_steps_on_pools_past_32_bits():
    """Slots whose states lie past 2^31 and 2^32 elements of their pool give what the same states give in a small one."""
    B, D, N, W = 5, 4096, 16, 4
    slots = [69999, 0, 65536, 32768, -1]
    s, c = scan_inputs("bf16", B, 1, D, N, 1), conv_inputs("bf16", B, 1, D, W, True)
    for pool_of, per, step in (
            (lambda n: torch.empty(n, D, N, device=DEV), s["initial_state"],
             lambda pool, n: pn.ssm_step(s["x"][:, 0], s["dt"][:, 0], s["A"], s["b"][:, 0], s["c"][:, 0], pool, gate=s["gate"][:, 0], slots=n)),
            (lambda n: torch.empty(n * 6, W - 1, D, device=DEV, dtype=torch.bfloat16), c["initial_state"],
             lambda pool, n: pn.short_conv_step(c["x"][:, 0], c["weight"], pool, bias=c["bias"], slots=n))):
        few = per.clone()
        want = step(few, torch.tensor([0, 1, 2, 3, -1], dtype=torch.int32, device=DEV))
        pool = pool_of(70000)
        at = [i * (pool.shape[0] // 70000) for i in slots[:4]]
        for i, b in zip(at, range(4)):
            pool[i] = per[b]
        got = step(pool, torch.tensor(at + [-1], dtype=torch.int32, device=DEV))
        assert pool.numel() > 1 << 32 and torch.equal(got, want)
        assert all(torch.equal(pool[i], few[b]) for i, b in zip(at, range(4)))
        del pool


def test_sequences_more_than_32_bits_apart():
    """Sequences 2^32 elements apart in memory are as good as their copies."""
    B, T, D, N = 2, 20, 40, 16
    far = torch.empty((1 << 32) + 4096, dtype=torch.bfloat16, device=DEV)

    def apart(t):
        v = far.as_strided(t.shape, (1 << 32, *t.stride()[1:]))
        return v.copy_(t)

    s, c, n = scan_inputs("bf16", B, T, D, N, 1), conv_inputs("bf16", B, T, D, 4, True), norm_inputs("bf16", "bf16", (B, T), D)
    kw = dict(skip=s["skip"], dt_bias=s["dt_bias"], gate=s["gate"])
    calls = [("x", c, lambda a: pn.short_conv(a["x"], a["weight"], bias=a["bias"])),
             ("dy", c, lambda a: pn.short_conv_backward(a["dy"], a["x"], a["weight"], bias=a["bias"])),
             ("x", n, lambda a: pn.block_norm(a["x"], a["weight"], residual=a["residual"])),
             ("residual", n, lambda a: pn.block_norm(a["x"], a["weight"], residual=a["residual"])),
             ("dy", n, lambda a: pn.block_norm_backward(a["dy"], a["ds"], a["x"], a["weight"], residual=a["residual"]))]
    for k in ("x", "dt", "b", "c"):
        calls.append((k, s, lambda a: pn.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"], **kw)))
    for k in ("dy", "x", "b"):
        calls.append((k, s, lambda a: pn.ssm_scan_backward(a["dy"], a["x"], a["dt"], a["A"], a["b"], a["c"], **kw)))
    for k, a, f in calls:
        _same(f(dict(a, **{k: apart(a[k])})), f(a))


def test_tokens_past_32_bits():
    """One sequence of 2^32 and some elements: its last tokens are those of a call that starts shortly before them, whose state
    is forgotten by then (e^-2 a token and less; 100 tokens are 1e-86).  The scan rounds its segments apart: twice the
    rounding of bfloat16, and of the float32 sums 100 U of their magnitude, which a tenth of a rounding covers where the
    result is not a small difference: 2^-12 of the largest value is added."""
    D, T, tail = 4096, (1 << 20) + 40, 200
    x = torch.empty(1, T, D, dtype=torch.bfloat16, device=DEV).uniform_(-1.0, 1.0)
    end = x[:, -tail:].contiguous()
    w, bias = torch.rand(D, 4, device=DEV), torch.rand(D, device=DEV)
    y, last = pn.short_conv(x, w, bias=bias)
    few, few_last = pn.short_conv(end, w, bias=bias)
    assert torch.equal(y[:, -100:], few[:, -100:]) and torch.equal(last, few_last)
    del y
    dx = pn.short_conv_backward(x, x, w, bias=bias)[0]
    assert torch.equal(dx[:, -100:], pn.short_conv_backward(end, end, w, bias=bias)[0][:, -100:])
    del dx
    y, s = pn.block_norm(x, bias, post_weight=bias)
    few, few_s = pn.block_norm(end, bias, post_weight=bias)
    assert torch.equal(y[:, -tail:], few) and torch.equal(s[:, -tail:], few_s)
    del y, s
    dx = pn.block_norm_backward(x, None, x, bias, post_weight=bias)[0]
    assert torch.equal(dx[:, -tail:], pn.block_norm_backward(end, None, end, bias, post_weight=bias)[0])
    del dx

    def close(got, want):
        got, want = got[:, -100:].float(), want[:, -100:].float()
        assert bool(((got - want).abs() <= 2.0 ** -7 * want.abs() + 2.0 ** -12 * want.abs().max()).all())

    A = -1.0 - torch.rand(D, 1, device=DEV)
    b = torch.rand(1, T, 1, 1, device=DEV).to(torch.bfloat16)
    args = lambda x, b: (x, x, A, b, b)  # noqa: E731
    dt_bias = torch.full((D,), 3.0, device=DEV)               # steps of 2.1 to 4.02
    end_b = b[:, -tail:].contiguous()
    close(pn.ssm_scan(*args(x, b), dt_bias=dt_bias)[0], pn.ssm_scan(*args(end, end_b), dt_bias=dt_bias)[0])
    got = pn.ssm_scan_backward(x, *args(x, b), dt_bias=dt_bias)
    want = pn.ssm_scan_backward(end, *args(end, end_b), dt_bias=dt_bias)
    close(got[0], want[0])
    close(got[1], want[1])


# ---------------------------------------------------------------- captured, and where a NaN goes


@pytest.mark.parametrize("N", [64, 128])
def test_scan_gradients_of_many_states_are_captured(N):
    """Workgroups of four and eight waves, whose LDS is more than a launch has by itself."""
    a = scan_inputs("bf16", 2, 90, 40, N, 1)

    def call():
        return pn.ssm_scan_backward(a["dy"], a["x"], a["dt"], a["A"], a["b"], a["c"], skip=a["skip"], gate=a["gate"],
                                    dt_bias=a["dt_bias"], initial_state=a["initial_state"], d_final_state=a["d_final_state"])

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for i in range(4):
        a["dy"].mul_(-0.75)
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        _same(out, want)


@pytest.mark.parametrize("N", [4, 16, 40])
@pytest.mark.parametrize("T", [30, 300])
@pytest.mark.parametrize("what", ["x", "dt", "gate", "b", "c"])
def test_scan_nans_stay_where_they_belong(N, T, what):
    """A NaN in a token of a channel (of a group, for b and c) reaches no earlier output, no other channel and no other
    sequence."""
    B, D, G, at = 2, 70, 2, T // 2
    a = scan_inputs("f32", B, T, D, N, G)
    kw = dict(skip=a["skip"], dt_bias=a["dt_bias"])

    def call():
        return pn.ssm_scan(a["x"], a["dt"], a["A"], a["b"], a["c"], gate=a["gate"], **kw)

    y, h = call()
    a[what][1, at, 1] = float("nan")
    bad = slice(1, 2) if what in ("x", "dt", "gate") else slice(D // G, D)
    got, state = call()
    reached = torch.zeros(B, T, D, dtype=torch.bool, device=DEV)
    reached[1, at:at + 1 if what in ("gate", "c") else T, bad] = True
    assert torch.equal(torch.isnan(got), reached) and torch.equal(torch.where(reached, 0, got), torch.where(reached, 0, y))
    left = torch.zeros(B, D, N, dtype=torch.bool, device=DEV)
    left[1, bad] = what not in ("gate", "c")
    assert torch.equal(torch.isnan(state), left) and torch.equal(torch.where(left, 0, state), torch.where(left, 0, h))
