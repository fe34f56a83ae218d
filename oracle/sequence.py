"""Sequence-layer operators in float64, from their definitions: rotary positions, norm + rotation, and linear attention
with a decay per head as the token-by-token recurrence, each with its gradients.

Token arrays are [B, T, heads, channels], states [B, H, dk, dv]; head h of H reads key and value head h // (H // HK).
"""

import numpy as np


def angles(positions, frequencies, magnitude=1.0):
    """(cos, sin) [..., R/2] of positions * frequencies."""
    a = np.asarray(positions, np.float64)[..., None] * np.asarray(frequencies, np.float64)
    return magnitude * np.cos(a), magnitude * np.sin(a)


def _pairs(R, interleaved):
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)


def rotate(x, cos, sin, interleaved=False):
    """x [B, T, H, D] turned by cos, sin [B, T, R/2]."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    ia, ib = _pairs(2 * cos.shape[-1], interleaved)
    c, s = cos[:, :, None], sin[:, :, None]
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def rotate_bound(x, cos, sin, interleaved=False):
    """Sum of the absolute values of the terms of each element of rotate()."""
    x = np.abs(np.asarray(x, np.float64))
    y = x.copy()
    ia, ib = _pairs(2 * cos.shape[-1], interleaved)
    c, s = np.abs(cos[:, :, None]), np.abs(sin[:, :, None])
    y[..., ia] = x[..., ia] * c + x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def norm(x, w, eps):
    """(w x r, r) with r = (mean x^2 + eps)^{-1/2} over the channels."""
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return x * r * (1.0 if w is None else np.asarray(w, np.float64)), r


def norm_rotate_backward(dy, x, w, cos, sin, eps, interleaved=False):
    """(dx, dw per head [H, D]) of rotate(norm(x)), and the sums of absolute terms of both."""
    x = np.asarray(x, np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, np.float64)
    g = rotate(dy, cos, -sin, interleaved)
    ga = rotate_bound(dy, cos, sin, interleaved)
    _, r = norm(x, None, eps)
    n = x * r
    e = g * w
    dx = r * (e - n * np.mean(e * n, axis=-1, keepdims=True))
    bx = r * (ga * np.abs(w) + np.abs(n) * np.mean(ga * np.abs(w * n), axis=-1, keepdims=True))
    return dx, np.sum(g * n, axis=(0, 1)), bx, np.sum(ga * np.abs(n), axis=(0, 1))


def _share(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[2], axis=2)


def linear_attention(q, k, v, log_decay, initial_state=None, scale=1.0, lengths=None):
    """(o, final state) of S_t = lam S_{t-1} + k_t^T v_t, o_t = scale q_t S_t."""
    B, T, H, DK = q.shape
    q, k, v = np.asarray(q, np.float64), _share(k, H), _share(v, H)
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    lam = np.exp(np.asarray(log_decay, np.float64))
    o = np.zeros((B, T, H, v.shape[-1]))
    S = np.zeros((B, H, DK, v.shape[-1])) if initial_state is None else np.array(initial_state, np.float64)
    for b in range(B):
        for t in range(n[b]):
            S[b] = lam[:, None, None] * S[b] + k[b, t, :, :, None] * v[b, t, :, None, :]
            o[b, t] = scale * np.einsum("hi,hij->hj", q[b, t], S[b])
    return o, S


def linear_attention_backward(do, q, k, v, log_decay, initial_state=None, d_final_state=None, scale=1.0, lengths=None):
    """(dq, dk, dv, d_initial_state): S forward in time, its gradient R backward."""
    B, T, H, DK = q.shape
    HK = k.shape[2]
    q, k, v, do = np.asarray(q, np.float64), _share(k, H), _share(v, H), np.asarray(do, np.float64)
    n = np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)
    lam = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    DV = v.shape[-1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    S = np.zeros((B, H, DK, DV)) if initial_state is None else np.array(initial_state, np.float64)
    R = np.zeros((B, H, DK, DV)) if d_final_state is None else np.array(d_final_state, np.float64)
    for b in range(B):
        for t in range(n[b]):
            S[b] = lam * S[b] + k[b, t, :, :, None] * v[b, t, :, None, :]
            dq[b, t] = scale * np.einsum("hij,hj->hi", S[b], do[b, t])
        for t in reversed(range(n[b])):
            R[b] = R[b] + scale * q[b, t, :, :, None] * do[b, t, :, None, :]
            dk[b, t] = np.einsum("hij,hj->hi", R[b], v[b, t])
            dv[b, t] = np.einsum("hi,hij->hj", k[b, t], R[b])
            R[b] = lam * R[b]
    join = lambda x: x.reshape(B, T, HK, H // HK, -1).sum(3)  # noqa: E731
    return dq, join(dk), join(dv), R
