"""State-space operators of libpn: the short causal convolution, the selective scan and the norms around a block
(include/pn.h holds the definitions, layouts and limits).

Argument marshalling only, in the manner of ``sequence.py``: token tensors are [B, T, channels] in float32, bfloat16 or
float16 with adjacent channels and any other strides, weights contiguous float32, states contiguous; every call enqueues on
the current stream of the tensors' device and returns without waiting; outputs are new contiguous tensors.  Gradients are
calls of their own (examples/state_space_layer.py wraps them in autograd functions).
"""

import ctypes
import struct

import torch

from .sequence import _DTYPES, _array, _raw_stream, _refuse, _run, _shape_is, _workspace

# Argument blocks of include/pn.h: every field is 8 bytes wide.
_CONV = struct.Struct("=6q3q4qq2q4qqq2qq3q").pack
_CONV_STEP = struct.Struct("=5q2q4q2qq2q").pack
_SSM = struct.Struct("=7q3qq20qqqq4qq5q3qq3q").pack
_SSM_STEP = struct.Struct("=6q3q20q3q2q").pack
_NORM = struct.Struct("=5qd3q12q2q8q3q3q3q").pack
_NONE = (0, 0, 0, 0)

EXPORTED = ("pn_short_conv", "pn_short_conv_backward", "pn_short_conv_workspace_bytes", "pn_short_conv_step", "pn_ssm_scan",
            "pn_ssm_scan_backward", "pn_ssm_scan_workspace_bytes", "pn_ssm_step", "pn_block_norm", "pn_block_norm_backward",
            "pn_block_norm_workspace_bytes")


def declare(L):
    """ctypes signatures of this part of the library."""
    for name in EXPORTED:
        f = getattr(L, name)
        size = name.endswith("_bytes")
        f.argtypes = [ctypes.c_char_p, ctypes.c_int32] if name == "pn_ssm_scan_workspace_bytes" else [ctypes.c_char_p]
        f.restype = ctypes.c_size_t if size else ctypes.c_int


def _strides(t, name):
    """(address, batch and token stride, 0) of tokens [B, T, D] or, one of each sequence, [B, D]."""
    s = t.stride()
    if s[-1] != 1 and t.shape[-1] != 1:
        raise ValueError(f"the channels of {name} must be adjacent (stride 1, got {s[-1]})")
    return (t.data_ptr(), s[0], s[1], 0) if len(s) == 3 else (t.data_ptr(), s[0], 0, 0)


def _first(t, name, *dims):
    """(shape, dtype, its code, device index, address and strides) of the tensor that the others have to agree with."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    dt = t.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dt}")
    shape = tuple(t.shape)
    if len(shape) not in dims:
        raise ValueError(f"{name} must have {' or '.join(map(str, dims))} dimensions, got shape {shape}")
    return shape, dt, code, t.get_device(), _strides(t, name)


def _rows(t, name, dtype, shape, index):
    """(address, strides) of further tokens; None: none."""
    if t is None:
        return _NONE
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, dtype, index)
    if t.shape != shape:
        _shape_is(t, name, shape)
    return _strides(t, name)


def _given(t, name):
    """A tensor that cannot be left out."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    return t


def _like(x, dtype):
    """A contiguous output shaped as x (empty_like takes two thirds of new_empty's time, but keeps strides)."""
    return torch.empty_like(x) if x.dtype is dtype and x.is_contiguous() else x.new_empty(x.shape, dtype=dtype)


def _at(t):
    return 0 if t is None else t.data_ptr()


# ---------------------------------------------------------------- short convolution


def _conv_inputs(x, weight, bias, dims):
    shape, dt, code, dev, tok = _first(x, "x", dims)
    W = _given(weight, "weight").shape[-1] if _given(weight, "weight").dim() == 2 else 0
    f32 = torch.float32
    return shape, dt, code, dev, tok, W, _array(weight, "weight", f32, (shape[-1], W), dev), _array(bias, "bias", f32, (shape[-1],), dev)


def short_conv(x, weight, bias=None, initial_state=None, lengths=None, activation=True):
    """y_t = act(bias + sum_k weight[:, k] x_{t-W+1+k}) of each channel of x [B, T, D]; act(v) = v sigmoid(v), or v.

    weight float32 [D, W], 1 <= W <= 8, bias float32 [D]; initial_state [B, W - 1, D] (x's type) holds the tokens before the
    first, the newest last (None: zeros).  ``lengths`` (int32 [B]) ends sequences early: later tokens are not read and give
    zero rows.  Returns (y [B, T, D], the last W - 1 tokens [B, W - 1, D])."""
    (B, T, D), dt, code, dev, tok, W, w, b = _conv_inputs(x, weight, bias, 3)
    s0 = _array(initial_state, "initial_state", dt, (B, W - 1, D), dev)
    n = _array(lengths, "lengths", torch.int32, (B,), dev)
    y, final = _like(x, dt), x.new_empty(B, max(W - 1, 0), D)
    _run(dev, "pn_short_conv", _CONV(code, B, T, D, W, bool(activation), w, b, n, *tok, s0, y.data_ptr(), final.data_ptr(), *_NONE,
                                     0, 0, 0, 0, 0, 0, 0, _raw_stream(dev)))
    return y, final


def short_conv_backward(dy, x, weight, bias=None, initial_state=None, d_final_state=None, lengths=None, activation=True):
    """Gradients of ``short_conv`` from those of y and (if given) of the final state: (dx, dweight, dbias,
    d_initial_state), None where the input is."""
    (B, T, D), dt, code, dev, tok, W, w, b = _conv_inputs(x, weight, bias, 3)
    s0 = _array(initial_state, "initial_state", dt, (B, W - 1, D), dev)
    n = _array(lengths, "lengths", torch.int32, (B,), dev)
    grad = _rows(_given(dy, "dy"), "dy", dt, (B, T, D), dev)
    df = _array(d_final_state, "d_final_state", dt, (B, W - 1, D), dev)
    dx, dw = _like(x, dt), torch.empty_like(weight)
    db = torch.empty_like(bias) if bias is not None else None
    d0 = torch.empty_like(initial_state) if initial_state is not None else None

    def block(ws, nbytes):
        return _CONV(code, B, T, D, W, bool(activation), w, b, n, *tok, s0, 0, 0, *grad, df, dx.data_ptr(), dw.data_ptr(), _at(db),
                     _at(d0), ws, nbytes, _raw_stream(dev))

    ws, at, size = _workspace(x, "pn_short_conv_workspace_bytes", ("conv", code, B, T, D, W), block(0, 0))
    _run(dev, "pn_short_conv_backward", block(at, size))
    return dx, dw, db, d0


def short_conv_step(x, weight, state, bias=None, slots=None, activation=True):
    """One token x [B, D] of each sequence: returns y [B, D] and moves ``state`` [n_slots, W - 1, D] (x's type) on by it,
    sequence b at slots[b] (int32) or at b.  A slot outside the pool (by custom -1) marks an idle row: its y is 0 and
    nothing is updated.  Two rows must not name the same slot."""
    (B, D), dt, code, dev, tok, W, w, b = _conv_inputs(x, weight, bias, 2)
    n = _array(slots, "slots", torch.int32, (B,), dev)
    pool = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 3 else 0
    sp = _array(_given(state, "state"), "state", dt, (pool, W - 1, D), dev)
    y = _like(x, dt)
    _run(dev, "pn_short_conv_step", _CONV_STEP(code, B, D, W, bool(activation), w, b, *tok, sp, n, pool, y.data_ptr(), _raw_stream(dev)))
    return y


# ---------------------------------------------------------------- selective scan


def _ssm_inputs(x, dt, A, b, c, skip, gate, dt_bias, dims):
    shape, ty, code, dev, tok = _first(x, "x", dims)
    D, f32 = shape[-1], torch.float32
    N = _given(A, "A").shape[-1] if _given(A, "A").dim() == 2 else 0
    G = b.shape[-2] if isinstance(b, torch.Tensor) and b.dim() == dims + 1 else 0
    w = (_array(A, "A", f32, (D, N), dev), _array(skip, "skip", f32, (D,), dev), _array(dt_bias, "dt_bias", f32, (D,), dev))
    tok += _rows(_given(dt, "dt"), "dt", ty, shape, dev) + _rows(gate, "gate", ty, shape, dev)
    for t, name in ((b, "b"), (c, "c")):
        bc = (*shape[:-1], G, N)
        if not isinstance(t, torch.Tensor) or t.dtype is not ty or t.get_device() != dev:
            _refuse(t, name, ty, dev)
        if t.shape != bc:
            _shape_is(t, name, bc)
        s = t.stride()
        if s[-1] != 1 and N != 1:
            raise ValueError(f"the states of {name} must be adjacent (stride 1, got {s[-1]})")
        tok += (t.data_ptr(), s[0], s[1] if dims == 3 else 0, s[-2])
    return shape, ty, code, dev, N, G, w, tok


def ssm_scan(x, dt, A, b, c, skip=None, gate=None, dt_bias=None, softplus=True, initial_state=None, lengths=None):
    """h_t = exp(delta_t A) h_{t-1} + delta_t x_t b_t, y_t = (c_t . h_t + skip x_t) gate_t sigmoid(gate_t) of each channel,
    with delta = softplus(dt + dt_bias) (the plain sum without ``softplus``).

    x, dt and gate [B, T, D], A float32 [D, N] (1 <= N <= 128), b and c [B, T, G, N] (channel d reads group d / (D / G)),
    skip and dt_bias float32 [D], initial_state float32 [B, D, N] (None: zeros).  ``lengths`` (int32 [B]) ends sequences
    early: later tokens are not read and give zero rows.  Returns (y [B, T, D], final state float32 [B, D, N])."""
    (B, T, D), ty, code, dev, N, G, w, tok = _ssm_inputs(x, dt, A, b, c, skip, gate, dt_bias, 3)
    s0 = _array(initial_state, "initial_state", torch.float32, (B, D, N), dev)
    n = _array(lengths, "lengths", torch.int32, (B,), dev)
    y, final = _like(x, ty), A.new_empty(B, D, N)

    def block(ws, nbytes):
        return _SSM(code, B, T, D, N, G, bool(softplus), *w, n, *tok, s0, y.data_ptr(), final.data_ptr(), *_NONE, 0, 0, 0, 0, 0, 0,
                    0, 0, 0, 0, ws, nbytes, _raw_stream(dev))

    ws, at, size = _workspace(x, "pn_ssm_scan_workspace_bytes", ("scan", code, B, T, D, N, G), block(0, 0), 0)
    _run(dev, "pn_ssm_scan", block(at, size))
    return y, final


def ssm_scan_backward(dy, x, dt, A, b, c, skip=None, gate=None, dt_bias=None, softplus=True, initial_state=None,
                      d_final_state=None, lengths=None):
    """Gradients of ``ssm_scan`` from those of y and (if given) of the final state: (dx, ddt, dA, db, dc, dskip, dgate,
    ddt_bias, d_initial_state), None where the input is.  Takes a workspace of about 0.6 to 0.8 B T D N bytes."""
    (B, T, D), ty, code, dev, N, G, w, tok = _ssm_inputs(x, dt, A, b, c, skip, gate, dt_bias, 3)
    s0 = _array(initial_state, "initial_state", torch.float32, (B, D, N), dev)
    n = _array(lengths, "lengths", torch.int32, (B,), dev)
    grad = _rows(_given(dy, "dy"), "dy", ty, (B, T, D), dev)
    df = _array(d_final_state, "d_final_state", torch.float32, (B, D, N), dev)
    dx, ddt, db, dc = _like(x, ty), _like(x, ty), _like(b, ty), _like(b, ty)
    dz = _like(x, ty) if gate is not None else None
    dA, (dskip, dbias, d0) = torch.empty_like(A), (torch.empty_like(t) if t is not None else None
                                                   for t in (skip, dt_bias, initial_state))

    def block(ws, nbytes):
        return _SSM(code, B, T, D, N, G, bool(softplus), *w, n, *tok, s0, 0, 0, *grad, df, dx.data_ptr(), ddt.data_ptr(), _at(dz),
                    db.data_ptr(), dc.data_ptr(), dA.data_ptr(), _at(dskip), _at(dbias), _at(d0), ws, nbytes, _raw_stream(dev))

    ws, at, size = _workspace(x, "pn_ssm_scan_workspace_bytes", ("scan gradients", code, B, T, D, N, G), block(0, 0), 1)
    _run(dev, "pn_ssm_scan_backward", block(at, size))
    return dx, ddt, dA, db, dc, dskip, dz, dbias, d0


def ssm_step(x, dt, A, b, c, state, skip=None, gate=None, dt_bias=None, softplus=True, slots=None):
    """One token of each sequence: updates ``state`` float32 [n_slots, D, N] in place and returns y [B, D].

    x, dt and gate [B, D], b and c [B, G, N]; sequence b at slots[b] (int32) or at b.  A slot outside the pool (by custom
    -1) marks an idle row: its y is 0 and nothing is updated.  Two rows must not name the
    same slot."""
    (B, D), ty, code, dev, N, G, w, tok = _ssm_inputs(x, dt, A, b, c, skip, gate, dt_bias, 2)
    n = _array(slots, "slots", torch.int32, (B,), dev)
    pool = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 3 else 0
    sp = _array(_given(state, "state"), "state", torch.float32, (pool, D, N), dev)
    y = _like(x, ty)
    _run(dev, "pn_ssm_step", _SSM_STEP(code, B, D, N, G, bool(softplus), *w, *tok, sp, n, pool, y.data_ptr(), _raw_stream(dev)))
    return y


# ---------------------------------------------------------------- norms around a block


def _norm_inputs(x, weight, gate, post_weight, scale):
    shape, dt, code, dev, tok = _first(x, "x", 2, 3)
    B, T, D = shape if len(shape) == 3 else (shape[0], 1, shape[1])
    w = tuple(_array(t, name, torch.float32, (D,), dev)
              for t, name in ((weight, "weight"), (post_weight, "post_weight"), (scale, "scale")))
    return shape, (B, T, D), dt, code, dev, tok + _rows(gate, "gate", dt, shape, dev), w


def _residual_type(t, name, dt):
    """The type of a residual stream, that of the tokens or float32."""
    if _given(t, name).dtype not in (dt, torch.float32):
        raise TypeError(f"{name} must be {dt} or torch.float32, got {t.dtype}")
    return t.dtype


def block_norm(x, weight=None, residual=None, gate=None, post_weight=None, scale=None, eps=1e-6):
    """From what a block gave, x, to what the next one takes, y, over the residual stream: with u = x gate sigmoid(gate)
    (x without a gate) and p = u / sqrt(mean u^2 + eps) * post_weight (u without it),

        s = residual + scale * p,      y = s / sqrt(mean s^2 + eps) * weight.

    x and gate [B, T, D] or [B, D], residual the same in x's type or float32 (None: 0), weights and scale float32 [D].
    Returns (y, s), y None without ``weight``; s has the residual's type."""
    shape, sizes, dt, code, dev, tok, w = _norm_inputs(x, weight, gate, post_weight, scale)
    rt = dt if residual is None else _residual_type(residual, "residual", dt)
    res = _rows(residual, "residual", rt, shape, dev)
    y = _like(x, dt) if weight is not None else None
    s = _like(x, rt)
    _run(dev, "pn_block_norm", _NORM(code, _DTYPES[rt], *sizes, float(eps), *w, *tok, *res, _at(y), s.data_ptr(), *_NONE, *_NONE,
                                     0, 0, 0, 0, 0, 0, 0, 0, _raw_stream(dev)))
    return y, s


def block_norm_backward(dy, ds, x, weight=None, residual=None, gate=None, post_weight=None, scale=None, eps=1e-6):
    """Gradients of ``block_norm`` from those of y (None without ``weight``) and s (None: 0): (dx, dweight, dresidual, dgate,
    dpost_weight, dscale), None where the input is."""
    shape, sizes, dt, code, dev, tok, w = _norm_inputs(x, weight, gate, post_weight, scale)
    rt = dt if residual is None else _residual_type(residual, "residual", dt)
    res = _rows(residual, "residual", rt, shape, dev)
    gy = _rows(_given(dy, "dy"), "dy", dt, shape, dev) if weight is not None else _NONE
    gs = _rows(ds, "ds", rt, shape, dev)
    dx, dr = _like(x, dt), _like(x, rt) if residual is not None else None
    dz = _like(x, dt) if gate is not None else None
    dw, dpw, dsc = (torch.empty_like(t) if t is not None else None for t in (weight, post_weight, scale))

    def block(ws, nbytes):
        return _NORM(code, _DTYPES[rt], *sizes, float(eps), *w, *tok, *res, 0, 0, *gy, *gs, dx.data_ptr(), _at(dz), _at(dr),
                     _at(dw), _at(dpw), _at(dsc), ws, nbytes, _raw_stream(dev))

    key = ("norm", code, *sizes, weight is None, post_weight is None, scale is None)
    ws, at, size = _workspace(x, "pn_block_norm_workspace_bytes", key, block(0, 0))
    _run(dev, "pn_block_norm_backward", block(at, size))
    return dx, dw, dr, dz, dpw, dsc
