"""State-space operators in float64, from their definitions: the short causal convolution, the selective scan token by token
and the norms around a block, each with its gradients.

Tokens are [B, T, D], the scan's b and c [B, T, G, N], its states [B, D, N], the convolution's state the last W - 1 tokens
[B, W - 1, D].  The gradients also come as the sums of the absolute values of their terms, which error bounds are made of:
second results of short_conv_backward and block_norm_backward, ssm_scan_backward with ``bound``.
"""

import numpy as np


def _f(x):
    return None if x is None else np.asarray(x, np.float64)


def logistic(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def softplus(v):
    return np.maximum(v, 0.0) + np.log1p(np.exp(-np.abs(v)))


def _lengths(lengths, B, T):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths), 0, T)


# ---------------------------------------------------------------- short convolution


def _rows(x, past, n):
    """The tokens before the first and the n of the sequence: [W - 1 + n, D]."""
    return np.concatenate((past, x[:n]))


def short_conv(x, weight, bias=None, initial_state=None, lengths=None, activation=True):
    """(y, final state, y before the activation)."""
    x, weight = _f(x), _f(weight)
    B, T, D = x.shape
    W = weight.shape[1]
    y, pre, final = np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, W - 1, D))
    for b, n in enumerate(_lengths(lengths, B, T)):
        past = np.zeros((W - 1, D)) if initial_state is None else _f(initial_state)[b]
        rows = _rows(x[b], past, n)
        for t in range(n):
            pre[b, t] = (0.0 if bias is None else _f(bias)) + sum(weight[:, k] * rows[t + k] for k in range(W))
        y[b, :n] = pre[b, :n] * logistic(pre[b, :n]) if activation else pre[b, :n]
        final[b] = rows[n:]
    return y, final, pre


def short_conv_backward(dy, x, weight, bias=None, initial_state=None, d_final_state=None, lengths=None, activation=True):
    """((dx, dweight, dbias, d_initial_state), the same sums over absolute values)."""
    x, weight, dy = _f(x), _f(weight), _f(dy)
    B, T, D = x.shape
    W = weight.shape[1]
    pre = short_conv(x, weight, bias, initial_state, lengths, activation)[2]
    out = [[np.zeros((B, T, D)), np.zeros((D, W)), np.zeros(D), np.zeros((B, W - 1, D))] for _ in range(2)]
    for b, n in enumerate(_lengths(lengths, B, T)):
        past = np.zeros((W - 1, D)) if initial_state is None else _f(initial_state)[b]
        rows = _rows(x[b], past, n)
        p = logistic(pre[b, :n])
        d = dy[b, :n] * (p * (1.0 + pre[b, :n] * (1.0 - p)) if activation else 1.0)
        for (dx, dw, db, d0), f in zip(out, (lambda v: v, np.abs)):
            grad = np.zeros((W - 1 + n, D))
            if d_final_state is not None:
                grad[n:] += f(_f(d_final_state)[b])
            for t in range(n):
                for k in range(W):
                    grad[t + k] += f(weight[:, k] * d[t])
                    dw[:, k] += f(d[t] * rows[t + k])
                db += f(d[t])
            dx[b, :n], d0[b] = grad[W - 1:], grad[:W - 1]
    return tuple(out[0]), tuple(out[1])


# ---------------------------------------------------------------- selective scan


def _steps(dt, dt_bias, use):
    v = _f(dt) + (0.0 if dt_bias is None else _f(dt_bias))
    return (softplus(v), logistic(v)) if use else (v, np.ones_like(v))


def ssm_scan(x, dt, A, b, c, skip=None, gate=None, dt_bias=None, softplus=True, initial_state=None, lengths=None):
    """(y, final state)."""
    x, A, b, c = _f(x), _f(A), _f(b), _f(c)
    B, T, D = x.shape
    G, N = b.shape[2:]
    delta, _ = _steps(dt, dt_bias, softplus)
    b, c = np.repeat(b, D // G, 2), np.repeat(c, D // G, 2)
    h = np.zeros((B, D, N)) if initial_state is None else _f(initial_state).copy()
    y = np.zeros((B, T, D))
    for i, n in enumerate(_lengths(lengths, B, T)):
        for t in range(n):
            h[i] = np.exp(delta[i, t][:, None] * A) * h[i] + (delta[i, t] * x[i, t])[:, None] * b[i, t]
            y[i, t] = (c[i, t] * h[i]).sum(-1)
            if skip is not None:
                y[i, t] += _f(skip) * x[i, t]
            if gate is not None:
                z = _f(gate)[i, t]
                y[i, t] *= z * logistic(z)
    return y, h


def ssm_scan_backward(dy, x, dt, A, b, c, skip=None, gate=None, dt_bias=None, softplus=True, initial_state=None,
                      d_final_state=None, lengths=None, bound=False):
    """(dx, ddt, dA, db, dc, dskip, dgate, ddt_bias, d_initial_state): states forward in time, their gradients backward;
    with ``bound`` the sums of absolute terms."""
    x, A, dy = _f(x), _f(A), _f(dy)
    B, T, D = x.shape
    G, N = b.shape[2:]
    delta, slope = _steps(dt, dt_bias, softplus)
    f = np.abs if bound else (lambda v: v)
    bw, cw = np.repeat(_f(b), D // G, 2), np.repeat(_f(c), D // G, 2)
    skip = np.zeros(D) if skip is None else _f(skip)
    dx, ddt, dz = np.zeros((B, T, D)), np.zeros((B, T, D)), np.zeros((B, T, D))
    db, dc, dA, dskip = np.zeros((B, T, D, N)), np.zeros((B, T, D, N)), np.zeros((D, N)), np.zeros(D)
    d0 = np.zeros((B, D, N)) if d_final_state is None else f(_f(d_final_state).copy())
    for i, n in enumerate(_lengths(lengths, B, T)):
        h = np.zeros((D, N)) if initial_state is None else f(_f(initial_state)[i])
        states, kept = [], []
        for t in range(n):
            kept.append(np.exp(delta[i, t][:, None] * A) * h)
            h = kept[-1] + f((delta[i, t] * x[i, t])[:, None] * bw[i, t])
            states.append(h)
        r = d0[i]
        for t in reversed(range(n)):
            g = dy[i, t]
            if gate is not None:
                z = _f(gate)[i, t]
                p = logistic(z)
                y = (f(cw[i, t]) * states[t]).sum(-1) + f(skip * x[i, t])
                dz[i, t] = f(g * p * (1.0 + z * (1.0 - p))) * y
                g = g * z * p
            r = r + f(g[:, None] * cw[i, t])
            du = (r * f(bw[i, t])).sum(-1)
            w = r * kept[t]
            dd = f(x[i, t]) * du + (w * f(A)).sum(-1)
            dx[i, t] = f(delta[i, t]) * du + f(skip * g)
            ddt[i, t] = dd * slope[i, t]
            db[i, t] = r * f(delta[i, t] * x[i, t])[:, None]
            dc[i, t] = f(g)[:, None] * states[t]
            dA += w * f(delta[i, t])[:, None]
            dskip += f(g * x[i, t])
            r = np.exp(delta[i, t][:, None] * A) * r
        d0[i] = r
    join = lambda v: v.reshape(B, T, G, D // G, N).sum(3)  # noqa: E731
    return dx, ddt, dA, join(db), join(dc), dskip, dz, ddt.sum((0, 1)), d0


# ---------------------------------------------------------------- norms around a block


def block_norm(x, weight=None, residual=None, gate=None, post_weight=None, scale=None, eps=1e-6):
    """(y or None, s)."""
    u = _f(x) * (1.0 if gate is None else _f(gate) * logistic(_f(gate)))
    p = u if post_weight is None else u / np.sqrt((u * u).mean(-1, keepdims=True) + eps) * _f(post_weight)
    s = (0.0 if residual is None else _f(residual)) + (1.0 if scale is None else _f(scale)) * p
    return None if weight is None else s / np.sqrt((s * s).mean(-1, keepdims=True) + eps) * _f(weight), s


def block_norm_backward(dy, ds, x, weight=None, residual=None, gate=None, post_weight=None, scale=None, eps=1e-6):
    """((dx, dweight, dresidual, dgate, dpost_weight, dscale), the same sums over absolute values)."""
    x = _f(x)
    act, slope = 1.0, None
    if gate is not None:
        z = _f(gate)
        l = logistic(z)
        act, slope = z * l, l * (1.0 + z * (1.0 - l))
    u = x * act
    sc = 1.0 if scale is None else _f(scale)
    ru = 1.0 if post_weight is None else 1.0 / np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    res = 0.0 if residual is None else _f(residual)
    p = sc * u * ru * (1.0 if post_weight is None else _f(post_weight))
    lead = tuple(range(x.ndim - 1))
    both = []
    for f in (lambda v: v, np.abs):
        sign = -1.0 if f is not np.abs else 1.0
        t = np.zeros_like(x) if ds is None else f(_f(ds))
        dw = dpw = dsc = dz = None
        if weight is not None:
            s = res + p
            rs = 1.0 / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
            m, e = (f(res) + f(p)) * rs, f(_f(dy) * _f(weight))
            t = t + rs * (e + sign * m * (e * m).mean(-1, keepdims=True))
            dw = (f(_f(dy)) * m).sum(lead)
        dr, du = t, f(np.broadcast_to(sc, t.shape)) * t
        if post_weight is not None:
            n, pw = u * ru, _f(post_weight)
            dpw = (du * f(n)).sum(lead)
            dsc = (t * f(pw * n)).sum(lead)
            q = du * f(pw)
            du = ru * (q + sign * f(n) * (q * f(n)).mean(-1, keepdims=True))
        elif scale is not None:
            dsc = (t * f(u)).sum(lead)
        if gate is not None:
            dz = du * f(x * slope)
        both.append((du * f(np.broadcast_to(act, du.shape)), dw, dr if residual is not None else None, dz, dpw,
                     dsc if scale is not None else None))
    return tuple(both)
