"""Sequence-layer operators of libpn: rotary positions, norm + rotation of queries and keys, and linear attention with a
decay per head (include/pn.h holds the definitions, layouts and limits).

Argument marshalling only, as in the package's other entries.  Token tensors are [B, T, heads, channels] in float32,
bfloat16 or float16 with adjacent channels and any other strides (views of a packed projection need no copy); states are
contiguous float32 [B, H, dk, dv].  Every call enqueues on the current stream of the tensors' device and returns without
waiting; outputs are new contiguous tensors unless stated.  Gradients are calls of their own: nothing is recorded for
autograd (examples/sequence_layer.py wraps the calls in autograd functions).
"""

import ctypes
import math
import struct

import torch

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
# (a torch without device bindings has no tensors to call them for)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)

# Argument blocks of include/pn.h: every field is 8 bytes wide.
_ROTARY = struct.Struct("=9q8q2q3q4qd2q2q8q2q3q").pack
_ATTENTION = struct.Struct("=7qd2q12q3q4q5q3q").pack
_STEP = struct.Struct("=6qdq12q5q").pack
_NO_TOKENS = (0, 0, 0, 0)
_entries = {}            # entries of the loaded library
_sizes = {}              # workspace bytes by entry and sizes


def declare(L):
    """ctypes signatures of this part of the library."""
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    L.pn_rotary_table.argtypes = [vp, i64, i64, ctypes.c_double, vp, vp]
    for name in ("pn_rotary", "pn_qk_norm_rotary", "pn_qk_norm_rotary_backward", "pn_linear_attention",
                 "pn_linear_attention_backward", "pn_linear_attention_step"):
        getattr(L, name).argtypes = [ctypes.c_char_p]
        getattr(L, name).restype = ctypes.c_int
    L.pn_rotary_table.restype = ctypes.c_int
    L.pn_qk_norm_rotary_workspace_bytes.argtypes = [ctypes.c_char_p]
    L.pn_qk_norm_rotary_workspace_bytes.restype = ctypes.c_size_t
    L.pn_linear_attention_workspace_bytes.argtypes = [ctypes.c_char_p, i32]
    L.pn_linear_attention_workspace_bytes.restype = ctypes.c_size_t


EXPORTED = ("pn_rotary_table", "pn_rotary", "pn_qk_norm_rotary", "pn_qk_norm_rotary_backward",
            "pn_qk_norm_rotary_workspace_bytes", "pn_linear_attention", "pn_linear_attention_backward",
            "pn_linear_attention_workspace_bytes", "pn_linear_attention_step")


def _entry(name):
    from . import lib
    fn = getattr(lib(), name)
    _entries[name] = fn
    return fn


def _fail(rc):
    from . import PnError, last_error
    raise PnError(rc, last_error())


def _run(index, name, *args):
    """Call an entry on the device of its tensors."""
    fn = _entries.get(name) or _entry(name)
    if index == _current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc < 0:
        _fail(rc)


def _workspace(like, name, key, *args):
    """(tensor, address, bytes) of a 256-byte aligned workspace; the size is asked for once for the sizes in ``key``."""
    n = _sizes.get(key)
    if n is None:
        n = (_entries.get(name) or _entry(name))(*args)
        if n == 0:                                       # refused, as the call itself will be, which tells why
            return None, 0, 0
        if len(_sizes) >= 4096:
            _sizes.clear()
        _sizes[key] = n
    if n <= 256:                                         # none needed
        return None, 0, 0
    ws = torch.empty(n + 256, dtype=torch.uint8, device=like.device)
    return ws, (ws.data_ptr() + 255) & -256, n


# The checks below are written for calls of a few microseconds: each property is read once, and only a check that has
# failed looks for the reason.


def _refuse(t, name, dtype, index, contiguous=False):
    """The reason why a tensor is not on the device, of the type or (if asked) contiguous."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if contiguous and not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")
    raise ValueError(f"{name} must be on cuda:{index}")


def _shape_is(t, name, *shapes):
    raise ValueError(f"{name} must have shape {' or '.join(str(tuple(s)) for s in shapes)}, got {tuple(t.shape)}")


def _strides(t, name, shape):
    """(address, batch, token and head stride) of a token tensor of the right shape, whose channels have to be adjacent."""
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"the channels of {name} must be adjacent (stride 1, got {s[-1]})")
    return (t.data_ptr(), s[0], s[1], s[2]) if len(s) == 4 else (t.data_ptr(), s[0], 0, s[1])


def _tokens(t, name, shape, dtype, index):
    """(address, strides) of a token tensor; raises on what the library cannot take."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
        _refuse(t, name, dtype, index)
    if t.shape != shape:
        _shape_is(t, name, shape)
    return _strides(t, name, shape)


def _array(t, name, dtype, shape, index):
    """Address of a contiguous array (None: 0)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _refuse(t, name, dtype, index, True)
    if t.shape != shape:
        _shape_is(t, name, shape)
    return t.data_ptr()


def _first(t, name, dims):
    """(shape, dtype, its code, device index, address and strides) of the tensor that the others have to agree with."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    dt = t.dtype
    code = _DTYPES.get(dt)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dt}")
    shape = tuple(t.shape)
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {shape}")
    return shape, dt, code, t.get_device(), _strides(t, name, shape)


# ---------------------------------------------------------------- rotary positions


def rotary_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_positions=None, low=1.0, high=32.0):
    """Angles per position of the rotary_dim / 2 channel pairs, base^(-2i / rotary_dim), for contexts ``factor`` times longer
    than the ``original_positions`` a model was made for, scaled by

    "none"      nothing;
    "linear"    positions squeezed: every angle divided by factor;
    "base"      a larger base, base * factor^(R / (R - 2)): the slowest pair is divided by factor, the fastest kept;
    "by_parts"  by the turns a pair makes over the original context: more than ``high`` keep their angle, fewer than
                ``low`` are divided by factor, those between are mixed linearly in the number of turns.
    """
    R = int(rotary_dim)
    if R < 2 or R % 2 or R > 256:
        raise ValueError("rotary_dim must be even, 2 to 256")
    if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
        raise ValueError("base and factor must be positive and finite")
    if scaling == "base":
        if R < 4:
            raise ValueError('scaling "base" needs at least two pairs')
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if scaling in ("none", "base"):
        return f
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling != "by_parts":
        raise ValueError(f"unknown scaling {scaling!r}")
    if original_positions is None or not original_positions > 0:
        raise ValueError('scaling "by_parts" needs original_positions')
    if not low < high:
        raise ValueError("low must be below high")
    out = []
    for x in f:
        turns = original_positions * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - low) / (high - low)))
        out.append(x * keep + x / factor * (1.0 - keep))
    return out


def rotary_table(n_pos, frequencies, magnitude=1.0, device="cuda"):
    """[n_pos, R/2, 2] float32: magnitude * (cos, sin) of position * frequency, from float64; made once and kept."""
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("the table lives on a CUDA (HIP) device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    f = [float(x) for x in frequencies]
    table = torch.empty((int(n_pos), len(f), 2), dtype=torch.float32, device=device)
    _run(device.index, "pn_rotary_table", (ctypes.c_double * max(1, len(f)))(*f), len(f), int(n_pos), float(magnitude),
         table.data_ptr(), _raw_stream(device.index))
    return table


def _positions(positions, B, T, index):
    """(address, is int64, batch stride, token stride) of positions [B, T] or [T]."""
    if positions is None:
        return 0, 0, 0, 0
    dt = positions.dtype if isinstance(positions, torch.Tensor) else None
    if dt is not torch.int32 and dt is not torch.int64 or positions.get_device() != index:
        if dt is None or not positions.is_cuda or dt not in (torch.int32, torch.int64):
            raise TypeError("positions must be an int32 or int64 CUDA (HIP) tensor")
        raise ValueError(f"positions must be on cuda:{index}")
    s = positions.stride()
    if positions.shape == (B, T):
        return positions.data_ptr(), dt is torch.int64, s[0], s[1]
    if positions.shape == (T,):
        return positions.data_ptr(), dt is torch.int64, 0, s[0]
    _shape_is(positions, "positions", (B, T), (T,))


def _table(table, D, index):
    if (not isinstance(table, torch.Tensor) or table.dtype is not torch.float32 or table.get_device() != index or
            not table.is_contiguous()):
        _refuse(table, "table", torch.float32, index, True)
    shape = table.shape
    if len(shape) != 3 or shape[2] != 2 or 2 * shape[1] > D:
        raise ValueError(f"table must be [positions, R/2, 2] with R <= {D}, got {tuple(shape)}")
    return table.data_ptr(), shape[0], 2 * shape[1]


def _weight(w, name, heads, D, index):
    """(address, head stride) of a norm's weight [D] or [heads, D]; None: ones."""
    if w is None:
        return 0, 0
    if not isinstance(w, torch.Tensor) or w.dtype is not torch.float32 or w.get_device() != index or not w.is_contiguous():
        _refuse(w, name, torch.float32, index, True)
    if w.shape == (D,):
        return w.data_ptr(), 0
    if w.shape == (heads, D):
        return w.data_ptr(), D
    _shape_is(w, name, (D,), (heads, D))


def rotary(x, table, positions=None, offset=0, interleaved=False, inverse=False, out=None):
    """Turn the channel pairs of x [B, T, heads, D] by the angles of table row positions[b, t] (or offset + t).

    The first R = 2 * table.shape[1] channels rotate, as pairs (i, i + R/2), or (2i, 2i + 1) if ``interleaved``; the others
    pass.  ``inverse`` turns back: the gradient of the forward turn.  ``out`` may be x itself (contiguous)."""
    shape, dt, code, dev, tok = _first(x, "x", 4)
    B, T, H, D = shape
    tp, n_pos, R = _table(table, D, dev)
    pp, p64, psb, pst = _positions(positions, B, T, dev)
    if out is None:
        out = x.new_empty(B, T, H, D)
    else:
        _array(out, "out", dt, shape, dev)
    _run(dev, "pn_rotary", _ROTARY(
        code, B, T, D, R, bool(interleaved), bool(inverse), H, 0, *tok, *_NO_TOKENS, out.data_ptr(), 0, tp, n_pos, pp, p64,
        psb, pst, int(offset), 0.0, 0, 0, 0, 0, *_NO_TOKENS, *_NO_TOKENS, 0, 0, 0, 0, _raw_stream(dev)))
    return out


def _norm_inputs(q, k, q_weight, k_weight, table, positions):
    shape, dt, code, dev, tok = _first(q, "q", 4)
    B, T, H, D = shape
    HK = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
    kshape = (B, T, HK, D)
    tok += _tokens(k, "k", kshape, dt, dev)
    tp, n_pos, R = _table(table, D, dev)
    pos = _positions(positions, B, T, dev)
    qw, qs = _weight(q_weight, "q_weight", H, D, dev)
    kw, ks = _weight(k_weight, "k_weight", HK, D, dev)
    return dt, code, dev, shape, kshape, R, tok, (tp, n_pos, *pos), (qw, kw, qs, ks)


def qk_norm_rotary(q, k, q_weight, k_weight, table, positions=None, offset=0, eps=1e-6, interleaved=False):
    """Norm of each head of q [B, T, H, D] and k [B, T, HK, D] over its channels, times its float32 weight ([D], one per
    head [heads, D], or None), then the rotation of ``rotary``, in one pass.  Returns (q', k')."""
    dt, code, dev, shape, kshape, R, tok, at, w = _norm_inputs(q, k, q_weight, k_weight, table, positions)
    B, T, H, D = shape
    qo, ko = q.new_empty(*shape), q.new_empty(*kshape)
    _run(dev, "pn_qk_norm_rotary", _ROTARY(
        code, B, T, D, R, bool(interleaved), 0, H, kshape[2], *tok, qo.data_ptr(), ko.data_ptr(), *at, int(offset), float(eps),
        *w, *_NO_TOKENS, *_NO_TOKENS, 0, 0, 0, 0, _raw_stream(dev)))
    return qo, ko


def qk_norm_rotary_backward(dq_out, dk_out, q, k, q_weight, k_weight, table, positions=None, offset=0, eps=1e-6,
                            interleaved=False):
    """Gradients of ``qk_norm_rotary`` from those of its outputs: (dq, dk, dq_weight, dk_weight), a weight's gradient
    None where the weight is."""
    dt, code, dev, shape, kshape, R, tok, at, w = _norm_inputs(q, k, q_weight, k_weight, table, positions)
    B, T, H, D = shape
    grad = _tokens(dq_out, "dq_out", shape, dt, dev) + _tokens(dk_out, "dk_out", kshape, dt, dev)
    dq, dk = q.new_empty(*shape), q.new_empty(*kshape)
    dqw = torch.empty_like(q_weight) if w[0] else None
    dkw = torch.empty_like(k_weight) if w[1] else None

    def block(ws, nbytes):
        return _ROTARY(
            code, B, T, D, R, bool(interleaved), 0, H, kshape[2], *tok, dq.data_ptr(), dk.data_ptr(), *at, int(offset),
            float(eps), *w, *grad, dqw.data_ptr() if w[0] else 0, dkw.data_ptr() if w[1] else 0, ws, nbytes, _raw_stream(dev))

    ws, base, n = _workspace(q, "pn_qk_norm_rotary_workspace_bytes", (0, B, T, H, kshape[2], D), block(0, 0))
    _run(dev, "pn_qk_norm_rotary_backward", block(base, n))
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- linear attention


def _attention_inputs(q, k, v, log_decay, dims):
    shape, dt, code, dev, tok = _first(q, "q", dims)
    for t, name in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions")
    lead, HK, DV = shape[:-2], k.shape[-2], v.shape[-1]
    tok += _tokens(k, "k", (*lead, HK, shape[-1]), dt, dev) + _tokens(v, "v", (*lead, HK, DV), dt, dev)
    return shape, HK, DV, dt, code, dev, tok, _array(log_decay, "log_decay", torch.float32, (shape[-2],), dev)


def _scale(scale, channels):
    return float(scale) if scale is not None else channels ** -0.5 if channels else 1.0        # no channels: the library refuses them


def linear_attention(q, k, v, log_decay, initial_state=None, scale=None, lengths=None):
    """o_t = scale * q_t S_t with S_t = exp(log_decay) S_{t-1} + k_t^T v_t, for all T tokens.

    q [B, T, H, dk], k [B, T, HK, dk], v [B, T, HK, dv] (head h reads key and value head h / (H / HK)), log_decay float32
    [H], initial_state float32 [B, H, dk, dv] or None (zeros), scale dk^-1/2 by default.  ``lengths`` (int32 [B]) ends
    sequences early: later tokens are not read and give zero rows.  Returns (o [B, T, H, dv], final state float32)."""
    (B, T, H, DK), HK, DV, dt, code, dev, tok, g = _attention_inputs(q, k, v, log_decay, 4)
    s0 = _array(initial_state, "initial_state", torch.float32, (B, H, DK, DV), dev)
    n = _array(lengths, "lengths", torch.int32, (B,), dev)
    o = q.new_empty(B, T, H, DV)
    final = log_decay.new_empty(B, H, DK, DV)
    a = _scale(scale, DK)

    def block(ws, nbytes):
        return _ATTENTION(code, B, T, H, HK, DK, DV, a, g, n, *tok, s0, o.data_ptr(), final.data_ptr(), *_NO_TOKENS, 0, 0, 0,
                          0, 0, ws, nbytes, _raw_stream(dev))

    ws, at, size = _workspace(q, "pn_linear_attention_workspace_bytes", (1, code, B, T, H, HK, DK, DV), block(0, 0), 0)
    _run(dev, "pn_linear_attention", block(at, size))
    return o, final


def linear_attention_backward(do, q, k, v, log_decay, initial_state=None, d_final_state=None, scale=None, lengths=None):
    """Gradients of ``linear_attention`` from those of o and (if given) of the final state: (dq, dk, dv,
    d_initial_state), the last None without an initial state.  The decay is a constant."""
    (B, T, H, DK), HK, DV, dt, code, dev, tok, g = _attention_inputs(q, k, v, log_decay, 4)
    s0 = _array(initial_state, "initial_state", torch.float32, (B, H, DK, DV), dev)
    n = _array(lengths, "lengths", torch.int32, (B,), dev)
    td = _tokens(do, "do", (B, T, H, DV), dt, dev)
    df = _array(d_final_state, "d_final_state", torch.float32, (B, H, DK, DV), dev)
    dq, dk, dv = q.new_empty(B, T, H, DK), q.new_empty(B, T, HK, DK), q.new_empty(B, T, HK, DV)
    d0 = torch.empty_like(initial_state) if s0 else None
    a = _scale(scale, DK)

    def block(ws, nbytes):
        return _ATTENTION(code, B, T, H, HK, DK, DV, a, g, n, *tok, s0, 0, 0, *td, df, dq.data_ptr(), dk.data_ptr(),
                          dv.data_ptr(), d0.data_ptr() if s0 else 0, ws, nbytes, _raw_stream(dev))

    ws, at, size = _workspace(q, "pn_linear_attention_workspace_bytes", (2, code, B, T, H, HK, DK, DV), block(0, 0), 1)
    _run(dev, "pn_linear_attention_backward", block(at, size))
    return dq, dk, dv, d0


def linear_attention_step(q, k, v, log_decay, state, slots=None, scale=None):
    """One token of each sequence: updates ``state`` in place and returns o [B, H, dv].

    q [B, H, dk], k [B, HK, dk], v [B, HK, dv]; state float32 [n_slots, H, dk, dv], sequence b at slots[b] (int32) or at b.
    A slot outside the pool (by custom -1) marks an idle row: its o is 0 and nothing is updated."""
    (B, H, DK), HK, DV, dt, code, dev, tok, g = _attention_inputs(q, k, v, log_decay, 3)
    n = _array(slots, "slots", torch.int32, (B,), dev)
    pool = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 4 else 0
    sp = _array(state, "state", torch.float32, (pool, H, DK, DV), dev)
    o = q.new_empty(B, H, DV)
    _run(dev, "pn_linear_attention_step", _STEP(
        code, B, H, HK, DK, DV, _scale(scale, DK), g, *tok, sp, n, pool, o.data_ptr(),
        _raw_stream(dev)))
    return o
