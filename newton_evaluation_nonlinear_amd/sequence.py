"""Sequence-layer operators of libpn: rotary positions, norm + rotation of queries and keys, and linear attention with a
decay per head (include/pn.h holds the definitions, layouts and limits).

Argument marshalling only, as in the package's other entries.  Token tensors are [B, T, heads, channels] in float32,
bfloat16 or float16 with adjacent channels and any other strides (views of a packed projection need no copy); states are
contiguous float32 [B, H, dk, dv].  Every call enqueues on the current stream of the tensors' device and returns without
waiting; outputs are new contiguous tensors unless stated.
"""

import ctypes
import math
import struct

import torch

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_raw_stream = torch.cuda.current_stream

# Argument blocks of include/pn.h: every field is 8 bytes wide.
_ROTARY = struct.Struct("=9q8q2q3q4qd2q2q8q2q3q")
_ATTENTION = struct.Struct("=7qd2q12q3q4q5q3q")
_STEP = struct.Struct("=6qdq12q5q")
_NO_TOKENS = (0, 0, 0, 0)


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


def _run(device, name, *args):
    from . import PnError, last_error, lib
    fn = getattr(lib(), name)
    if device.index == torch.cuda.current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc < 0:
        raise PnError(rc, last_error())


def _workspace(device, name, *args):
    """A 256-byte aligned workspace of the size the entry asks for: (tensor, address, bytes)."""
    from . import EINVAL, PnError, last_error, lib
    n = getattr(lib(), name)(*args)
    if n == 0:
        raise PnError(EINVAL, last_error())
    ws = torch.empty(n + 256, dtype=torch.uint8, device=device)
    base = ws.data_ptr()
    aligned = (base + 255) // 256 * 256
    return ws, aligned, n


def _tokens(t, name, shape, dtype, device):
    """(address, strides) of a token tensor; raises on what the library cannot take."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    s = t.stride()
    if s[-1] != 1 and shape[-1] != 1:
        raise ValueError(f"the channels of {name} must be adjacent (stride 1, got {s[-1]})")
    return (t.data_ptr(), s[0], s[1], s[2]) if len(s) == 4 else (t.data_ptr(), s[0], 0, s[1])


def _array(t, name, dtype, shape, device):
    """Address of a contiguous array (None: 0)."""
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {dtype} CUDA (HIP) tensor")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    return t.data_ptr()


def _first(t, name, dims):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA (HIP) torch tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got shape {tuple(t.shape)}")
    return t.shape, t.dtype, t.device


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
    _run(device, "pn_rotary_table", (ctypes.c_double * max(1, len(f)))(*f), len(f), int(n_pos), float(magnitude),
         table.data_ptr(), _raw_stream(device).cuda_stream)
    return table


def _positions(positions, B, T, device):
    """(address, is int64, batch stride, token stride) of positions [B, T] or [T]."""
    if positions is None:
        return 0, 0, 0, 0
    if not isinstance(positions, torch.Tensor) or not positions.is_cuda or positions.dtype not in (torch.int32, torch.int64):
        raise TypeError("positions must be an int32 or int64 CUDA (HIP) tensor")
    if positions.device != device:
        raise ValueError(f"positions must be on {device}")
    s = positions.stride()
    if positions.shape == (B, T):
        sb, st = s
    elif positions.shape == (T,):
        sb, st = 0, s[0]
    else:
        raise ValueError(f"positions must have shape {(B, T)} or {(T,)}, got {tuple(positions.shape)}")
    return positions.data_ptr(), int(positions.dtype == torch.int64), sb, st


def _table(table, D, device):
    if not isinstance(table, torch.Tensor) or not table.is_cuda or table.dtype != torch.float32 or not table.is_contiguous():
        raise TypeError("table must be a contiguous float32 CUDA (HIP) tensor")
    if table.dim() != 3 or table.shape[2] != 2 or 2 * table.shape[1] > D:
        raise ValueError(f"table must be [positions, R/2, 2] with R <= {D}, got {tuple(table.shape)}")
    if table.device != device:
        raise ValueError(f"table must be on {device}")
    return table.data_ptr(), table.shape[0], 2 * table.shape[1]


def _weight(w, name, heads, D, device):
    """(address, head stride) of a norm's weight [D] or [heads, D]; None: ones."""
    if w is None:
        return 0, 0
    if not isinstance(w, torch.Tensor) or not w.is_cuda or w.dtype != torch.float32 or not w.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 CUDA (HIP) tensor")
    if w.device != device:
        raise ValueError(f"{name} must be on {device}")
    if w.shape == (D,):
        return w.data_ptr(), 0
    if w.shape == (heads, D):
        return w.data_ptr(), D
    raise ValueError(f"{name} must have shape {(D,)} or {(heads, D)}, got {tuple(w.shape)}")


def rotary(x, table, positions=None, offset=0, interleaved=False, inverse=False, out=None):
    """Turn the channel pairs of x [B, T, heads, D] by the angles of table row positions[b, t] (or offset + t).

    The first R = 2 * table.shape[1] channels rotate, as pairs (i, i + R/2), or (2i, 2i + 1) if ``interleaved``; the others
    pass.  ``inverse`` turns back: the gradient of the forward turn.  ``out`` may be x itself (contiguous)."""
    (B, T, H, D), dt, dev = _first(x, "x", 4)
    tok = _tokens(x, "x", x.shape, dt, dev)
    tp, n_pos, R = _table(table, D, dev)
    pos = _positions(positions, B, T, dev)
    if out is None:
        out = torch.empty((B, T, H, D), dtype=dt, device=dev)
    else:
        _array(out, "out", dt, x.shape, dev)
    _run(dev, "pn_rotary", _ROTARY.pack(
        _DTYPES[dt], B, T, D, R, int(bool(interleaved)), int(bool(inverse)), H, 0, *tok, *_NO_TOKENS, out.data_ptr(), 0,
        tp, n_pos, pos[0], pos[1], pos[2], pos[3], int(offset), 0.0, 0, 0, 0, 0, *_NO_TOKENS, *_NO_TOKENS, 0, 0, 0, 0,
        _raw_stream(dev).cuda_stream))
    return out


def qk_norm_rotary(q, k, q_weight, k_weight, table, positions=None, offset=0, eps=1e-6, interleaved=False):
    """Norm of each head of q [B, T, H, D] and k [B, T, HK, D] over its channels, times its float32 weight ([D], one per
    head [heads, D], or None), then the rotation of ``rotary``, in one pass.  Returns (q', k')."""
    (B, T, H, D), dt, dev = _first(q, "q", 4)
    HK = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
    tq, tk = _tokens(q, "q", q.shape, dt, dev), _tokens(k, "k", (B, T, HK, D), dt, dev)
    tp, n_pos, R = _table(table, D, dev)
    pos = _positions(positions, B, T, dev)
    qw, qs = _weight(q_weight, "q_weight", H, D, dev)
    kw, ks = _weight(k_weight, "k_weight", HK, D, dev)
    qo = torch.empty((B, T, H, D), dtype=dt, device=dev)
    ko = torch.empty((B, T, HK, D), dtype=dt, device=dev)
    _run(dev, "pn_qk_norm_rotary", _ROTARY.pack(
        _DTYPES[dt], B, T, D, R, int(bool(interleaved)), 0, H, HK, *tq, *tk, qo.data_ptr(), ko.data_ptr(), tp, n_pos,
        pos[0], pos[1], pos[2], pos[3], int(offset), float(eps), qw, kw, qs, ks, *_NO_TOKENS, *_NO_TOKENS, 0, 0, 0, 0,
        _raw_stream(dev).cuda_stream))
    return qo, ko


def qk_norm_rotary_backward(dq_out, dk_out, q, k, q_weight, k_weight, table, positions=None, offset=0, eps=1e-6,
                            interleaved=False):
    """Gradients of ``qk_norm_rotary`` from those of its outputs: (dq, dk, dq_weight, dk_weight), a weight's gradient
    None where the weight is."""
    (B, T, H, D), dt, dev = _first(q, "q", 4)
    HK = k.shape[2] if isinstance(k, torch.Tensor) and k.dim() == 4 else 0
    tq, tk = _tokens(q, "q", q.shape, dt, dev), _tokens(k, "k", (B, T, HK, D), dt, dev)
    gq, gk = _tokens(dq_out, "dq_out", q.shape, dt, dev), _tokens(dk_out, "dk_out", k.shape, dt, dev)
    tp, n_pos, R = _table(table, D, dev)
    pos = _positions(positions, B, T, dev)
    qw, qs = _weight(q_weight, "q_weight", H, D, dev)
    kw, ks = _weight(k_weight, "k_weight", HK, D, dev)
    dq = torch.empty((B, T, H, D), dtype=dt, device=dev)
    dk = torch.empty((B, T, HK, D), dtype=dt, device=dev)
    dqw = torch.empty_like(q_weight) if qw else None
    dkw = torch.empty_like(k_weight) if kw else None

    def block(ws, nbytes):
        return _ROTARY.pack(
            _DTYPES[dt], B, T, D, R, int(bool(interleaved)), 0, H, HK, *tq, *tk, dq.data_ptr(), dk.data_ptr(), tp, n_pos,
            pos[0], pos[1], pos[2], pos[3], int(offset), float(eps), qw, kw, qs, ks, *gq, *gk, dqw.data_ptr() if qw else 0,
            dkw.data_ptr() if kw else 0, ws, nbytes, _raw_stream(dev).cuda_stream)

    ws, at, n = _workspace(dev, "pn_qk_norm_rotary_workspace_bytes", block(0, 0))
    _run(dev, "pn_qk_norm_rotary_backward", block(at, n))
    return dq, dk, dqw, dkw


# ---------------------------------------------------------------- linear attention


def _attention_inputs(q, k, v, log_decay, initial_state, lengths, dims):
    (*lead, H, DK), dt, dev = _first(q, "q", dims)
    for t, name in ((k, "k"), (v, "v")):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions")
    HK, DV = k.shape[-2], v.shape[-1]
    tok = (_tokens(q, "q", q.shape, dt, dev) + _tokens(k, "k", (*lead, HK, DK), dt, dev) +
           _tokens(v, "v", (*lead, HK, DV), dt, dev))
    g = _array(log_decay, "log_decay", torch.float32, (H,), dev)
    s0 = _array(initial_state, "initial_state", torch.float32, (lead[0], H, DK, DV), dev)
    n = _array(lengths, "lengths", torch.int32, (lead[0],), dev)
    return dt, dev, lead, H, HK, DK, DV, tok, g, s0, n


def linear_attention(q, k, v, log_decay, initial_state=None, scale=None, lengths=None):
    """o_t = scale * q_t S_t with S_t = exp(log_decay) S_{t-1} + k_t^T v_t, for all T tokens.

    q [B, T, H, dk], k [B, T, HK, dk], v [B, T, HK, dv] (head h reads key and value head h / (H / HK)), log_decay float32
    [H], initial_state float32 [B, H, dk, dv] or None (zeros), scale dk^-1/2 by default.  ``lengths`` (int32 [B]) ends
    sequences early: later tokens are not read and give zero rows.  Returns (o [B, T, H, dv], final state float32)."""
    dt, dev, (B, T), H, HK, DK, DV, tok, g, s0, n = _attention_inputs(q, k, v, log_decay, initial_state, lengths, 4)
    o = torch.empty((B, T, H, DV), dtype=dt, device=dev)
    final = torch.empty((B, H, DK, DV), dtype=torch.float32, device=dev)
    a = DK ** -0.5 if scale is None else float(scale)

    def block(ws, nbytes):
        return _ATTENTION.pack(_DTYPES[dt], B, T, H, HK, DK, DV, a, g, n, *tok, s0, o.data_ptr(), final.data_ptr(),
                               *_NO_TOKENS, 0, 0, 0, 0, 0, ws, nbytes, _raw_stream(dev).cuda_stream)

    ws, at, size = _workspace(dev, "pn_linear_attention_workspace_bytes", block(0, 0), 0)
    _run(dev, "pn_linear_attention", block(at, size))
    return o, final


def linear_attention_backward(do, q, k, v, log_decay, initial_state=None, d_final_state=None, scale=None, lengths=None):
    """Gradients of ``linear_attention`` from those of o and (if given) of the final state: (dq, dk, dv,
    d_initial_state), the last None without an initial state.  The decay is a constant."""
    dt, dev, (B, T), H, HK, DK, DV, tok, g, s0, n = _attention_inputs(q, k, v, log_decay, initial_state, lengths, 4)
    td = _tokens(do, "do", (B, T, H, DV), dt, dev)
    df = _array(d_final_state, "d_final_state", torch.float32, (B, H, DK, DV), dev)
    dq = torch.empty((B, T, H, DK), dtype=dt, device=dev)
    dk = torch.empty((B, T, HK, DK), dtype=dt, device=dev)
    dv = torch.empty((B, T, HK, DV), dtype=dt, device=dev)
    d0 = torch.empty_like(initial_state) if initial_state is not None else None
    a = DK ** -0.5 if scale is None else float(scale)

    def block(ws, nbytes):
        return _ATTENTION.pack(_DTYPES[dt], B, T, H, HK, DK, DV, a, g, n, *tok, s0, 0, 0, *td, df, dq.data_ptr(),
                               dk.data_ptr(), dv.data_ptr(), 0 if d0 is None else d0.data_ptr(), ws, nbytes,
                               _raw_stream(dev).cuda_stream)

    ws, at, size = _workspace(dev, "pn_linear_attention_workspace_bytes", block(0, 0), 1)
    _run(dev, "pn_linear_attention_backward", block(at, size))
    return dq, dk, dv, d0


def linear_attention_step(q, k, v, log_decay, state, slots=None, scale=None):
    """One token of each sequence: updates ``state`` in place and returns o [B, H, dv].

    q [B, H, dk], k [B, HK, dk], v [B, HK, dv]; state float32 [n_slots, H, dk, dv], sequence b at slots[b] (int32) or at b.
    A slot outside the pool (by custom -1) marks an idle row: its o is 0 and nothing is updated."""
    dt, dev, (B,), H, HK, DK, DV, tok, g, _, n = _attention_inputs(q, k, v, log_decay, None, slots, 3)
    pool = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 4 else 0
    sp = _array(state, "state", torch.float32, (pool, H, DK, DV), dev)
    o = torch.empty((B, H, DV), dtype=dt, device=dev)
    _run(dev, "pn_linear_attention_step", _STEP.pack(
        _DTYPES[dt], B, H, HK, DK, DV, DK ** -0.5 if scale is None else float(scale), g, *tok, sp, n, pool, o.data_ptr(),
        _raw_stream(dev).cuda_stream))
    return o
