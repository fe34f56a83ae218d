"""Cases of the state-space operators: short causal convolution, selective scan and the norms around a block, for prompts,
training and single tokens.

``own`` False computes each operator from elementary torch operations in float32; True calls the library's entry points.
Tokens are [B, T, channels]; the scan's b and c [B, T, groups, N]; its states [B, channels, N] float32; the convolution's
state the last W - 1 tokens [B, W - 1, channels] in the storage type.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # a batch of prompts; x is a view of one packed projection of x and gate
        dict(name="conv prompt bf16", op="conv", B=8, T=4096, D=2048, W=4, dtype="bf16", initial=False, ragged=False,
             train=False),
        # a small training pass in float32, odd sizes, ragged, from and to a carried state
        dict(name="conv train f32", op="conv", B=5, T=1021, D=515, W=3, dtype="f32", initial=True, ragged=True, train=True),
        # one token for each of 4 sequences: latency
        dict(name="conv step bf16", op="conv_step", B=4, D=2048, W=4, dtype="bf16", pool=8),
        # a short prompt that continues a kept state: latency
        dict(name="scan short bf16", op="scan", B=1, T=37, D=2048, N=16, G=1, dtype="bf16", initial=True, ragged=False,
             train=False),
        # one long prompt: little to do side by side but the time axis
        dict(name="scan long bf16", op="scan", B=1, T=65536, D=2048, N=16, G=1, dtype="bf16", initial=False, ragged=False,
             train=False),
        # a ragged batch in float32, an odd number of channels, two groups of b and c
        dict(name="scan ragged f32", op="scan", B=16, T=2047, D=1026, N=16, G=2, dtype="f32", initial=True, ragged=True,
             train=False),
        # a training pass: output and all gradients
        dict(name="scan train bf16", op="scan", B=8, T=4096, D=2048, N=16, G=1, dtype="bf16", initial=False, ragged=False,
             train=True),
        # a small training pass in float32, odd sizes, from and to a carried state
        dict(name="scan train f32", op="scan", B=3, T=777, D=200, N=12, G=1, dtype="f32", initial=True, ragged=False,
             train=True),
        # one token for each of 256 sequences, states in a larger pool
        dict(name="scan step bf16", op="scan_step", B=256, D=4096, N=16, G=1, dtype="bf16", pool=320),
        # one token for each of 4 sequences between two blocks: latency
        dict(name="norm decode bf16", op="norm", B=4, T=1, D=2048, dtype="bf16", residual="bf16", gate=False, post=False,
             scale=False, train=False),
        # a batch of prompts: gate and norm after a block, scaled residual, norm before the next
        dict(name="norm prompt bf16", op="norm", B=8, T=4096, D=2048, dtype="bf16", residual="bf16", gate=True, post=True,
             scale=True, train=False),
        # a training pass on a float32 residual stream, odd sizes
        dict(name="norm train bf16", op="norm", B=4, T=2047, D=2050, dtype="bf16", residual="f32", gate=True, post=True,
             scale=True, train=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_step", "scan", "scan", "scan", "scan_step", "norm", "norm"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op.endswith("step"):
        B, D = _log(rng, 1, 256), _log(rng, 16, 4096)
        case = dict(op=op, B=B, D=D, dtype=dtype, pool=B + rng.randrange(0, 64))
        if op == "conv_step":
            return dict(case, W=rng.choice([2, 3, 4, 4, 5, 8]))
        G = rng.choice([g for g in (1, 1, 2, 4) if D % g == 0])
        return dict(case, N=rng.choice([1, 4, 7, 8, 16, 16]), G=G)
    T = 1 if rng.random() < 0.1 else _log(rng, 2, 32768)
    if op == "norm":
        D = _log(rng, 16, 8192)
        T = min(T, (1 << 26) // D)
        B = rng.randint(1, max(1, min(64, (1 << 25) // (T * D))))
        return dict(op=op, B=B, T=T, D=D, dtype=dtype, residual=rng.choice(["f32", dtype]), gate=rng.random() < 0.5,
                    post=rng.random() < 0.6, scale=rng.random() < 0.5, train=rng.random() < 0.5)
    D = _log(rng, 16, 4096)
    train = rng.random() < 0.5
    case = dict(op=op, T=T, D=D, dtype=dtype, initial=rng.random() < 0.5, ragged=rng.random() < 0.4, train=train)
    if op == "conv":
        T = case["T"] = min(T, (1 << 26) // D)
        return dict(case, B=rng.randint(1, max(1, min(64, (1 << 25) // (T * D)))), W=rng.choice([1, 2, 3, 4, 4, 5, 8]))
    N = rng.choice([1, 4, 8, 12, 16, 16, 16, 24, 64])
    most = (1 << 28) if train else (1 << 30)             # elements of states over time
    while T * D * N > most:
        T = (T + 1) // 2
    G = rng.choice([g for g in (1, 1, 2, 4) if D % g == 0])
    return dict(case, T=T, B=rng.randint(1, max(1, min(16, most // (T * D * N)))), N=N, G=G)


def work(case):
    n = DTYPES[case["dtype"]].itemsize
    B, D, op = case["B"], case["D"], case["op"]
    if op == "conv_step":
        W = case["W"]
        return {"bytes": n * B * D * (2 + 2 * (W - 1)) + 4 * D * (W + 1), "flops": B * D * (2 * W + 4)}
    if op == "scan_step":
        N, G = case["N"], case["G"]
        return {"bytes": B * (8 * D * N + n * (4 * D + 2 * G * N)) + 4 * D * (N + 2), "flops": 7 * B * D * N}
    T = case["T"]
    if op == "norm":
        r = 4 if case["residual"] == "f32" else 2 if n == 2 else 4
        e = B * T * D
        w = 4 * D * (1 + case["post"] + case["scale"])
        if not case["train"]:
            return {"bytes": e * (n * (2 + case["gate"]) + 2 * r) + w, "flops": e * (6 + 4 * case["post"] + 6 * case["gate"])}
        back = n * (3 + 2 * case["gate"]) + 3 * r        # dy, x, dx, gate, dgate; ds, s, dresidual
        return {"bytes": e * (n * (2 + case["gate"]) + 2 * r + back) + 3 * w,
                "flops": 3 * e * (6 + 4 * case["post"] + 6 * case["gate"])}
    tokens = B * T * (3 if case["ragged"] else 4) // 4   # about the tokens that are read
    if op == "conv":
        W = case["W"]
        state = n * B * D * (W - 1) * (2 if case["initial"] else 1)
        if not case["train"]:
            return {"bytes": n * D * (tokens + B * T) + state + 4 * D * (W + 1), "flops": tokens * D * (2 * W + 4)}
        return {"bytes": n * D * (3 * tokens + 2 * B * T) + 2 * state + 12 * D * (W + 1),
                "flops": 3 * tokens * D * (2 * W + 4)}
    N, G = case["N"], case["G"]
    state = 4 * B * D * N * (2 if case["initial"] else 1)
    read = n * tokens * (3 * D + 2 * G * N) + 4 * D * (N + 2)
    if not case["train"]:
        return {"bytes": read + n * B * T * D + state, "flops": 7 * tokens * D * N}
    put = n * B * T * (4 * D + 2 * G * N) + 4 * D * (N + 2)
    return {"bytes": 2 * read + n * tokens * D + put + 2 * state, "flops": 23 * tokens * D * N}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, D, op = case["B"], case["D"], case["op"]

    def normal(*shape, to=dt, by=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * by).to(to)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    s = dict(case)
    f32 = torch.float32
    if op.endswith("step"):
        s["slots"] = torch.randperm(case["pool"], device="cuda", generator=g)[:B].to(torch.int32)
    if op in ("conv", "conv_step"):
        W = case["W"]
        s["weight"] = normal(D, W, to=f32, by=W ** -0.5)
        s["bias"] = normal(D, to=f32, by=0.2)
        if op == "conv_step":
            s["x"] = normal(B, 2 * D)[:, :D]
            s["state"] = normal(case["pool"], W - 1, D)
            return s
        T = case["T"]
        s["x"] = normal(B, T, 2 * D)[..., :D]
        s["initial"] = normal(B, W - 1, D) if case["initial"] else None
        if case["train"]:
            s["dy"] = normal(B, T, D)
            s["dfinal"] = normal(B, W - 1, D, by=0.5) if case["initial"] else None
    elif op in ("scan", "scan_step"):
        N, G = case["N"], case["G"]
        # decays 1 .. N per unit of time, varied from channel to channel, and steps of 0.001 to 0.1 about their bias
        s["A"] = -(torch.arange(1, N + 1, device="cuda") * torch.exp(0.2 * torch.randn(D, N, device="cuda", generator=g)))
        s["skip"] = 1.0 + normal(D, to=f32, by=0.2)
        step = torch.exp(uniform(D) * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        s["dt_bias"] = step + torch.log(-torch.expm1(-step))
        lead = (B,) if op == "scan_step" else (B, case["T"])
        s["x"], s["dt"], s["gate"] = normal(*lead, D), normal(*lead, D, by=0.5), normal(*lead, 2 * D)[..., D:]
        bc = normal(*lead, 2 * G * N)                    # one projection holds b and c
        s["b"], s["c"] = bc[..., :G * N].unflatten(-1, (G, N)), bc[..., G * N:].unflatten(-1, (G, N))
        if op == "scan_step":
            s["state"] = normal(case["pool"], D, N, to=f32)
            return s
        T = case["T"]
        s["initial"] = normal(B, D, N, to=f32) if case["initial"] else None
        if case["train"]:
            s["dy"] = normal(B, T, D)
            s["dfinal"] = normal(B, D, N, to=f32, by=0.5) if case["initial"] else None
    else:
        T = case["T"]
        rt = DTYPES[case["residual"]]
        s["x"], s["r"] = normal(B, T, D), normal(B, T, D, to=rt, by=2.0)
        s["gate_"] = normal(B, T, D) if case["gate"] else None
        s["w"] = 1.0 + normal(D, to=f32, by=0.2)
        s["pw"] = 1.0 + normal(D, to=f32, by=0.2) if case["post"] else None
        s["sc"] = normal(D, to=f32, by=0.5) if case["scale"] else None
        s["eps"] = 1e-6
        if case["train"]:
            s["dy"], s["ds"] = normal(B, T, D), normal(B, T, D, to=rt, by=0.5)
        return s
    s["lengths"] = (torch.randint(max(1, case["T"] // 2), case["T"] + 1, (B,), device="cuda", generator=g).to(torch.int32)
                    if case["ragged"] else None)
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"conv": _conv, "conv_step": _conv_step, "scan": _scan, "scan_step": _scan_step, "norm": _norm}[s["op"]](s)


def _run_own(s):
    import newton_evaluation_nonlinear_amd as pn

    op = s["op"]
    if op == "conv_step":
        return pn.short_conv_step(s["x"], s["weight"], s["state"], bias=s["bias"], slots=s["slots"]), s["state"]
    if op == "conv":
        kw = dict(bias=s["bias"], initial_state=s["initial"], lengths=s["lengths"])
        out = pn.short_conv(s["x"], s["weight"], **kw)
        if not s["train"]:
            return out
        back = pn.short_conv_backward(s["dy"], s["x"], s["weight"], d_final_state=s["dfinal"], **kw)
        return out + (back if s["initial"] is not None else back[:3])
    if op == "norm":
        kw = dict(gate=s["gate_"], post_weight=s["pw"], scale=s["sc"], eps=s["eps"])
        y, r = pn.block_norm(s["x"], s["w"], residual=s["r"], **kw)
        if not s["train"]:
            return y, r
        back = pn.block_norm_backward(s["dy"], s["ds"], s["x"], s["w"], residual=s["r"], **kw)
        return (y, r) + tuple(t for t in back if t is not None)
    kw = dict(skip=s["skip"], gate=s["gate"], dt_bias=s["dt_bias"])
    if op == "scan_step":
        return pn.ssm_step(s["x"], s["dt"], s["A"], s["b"], s["c"], s["state"], slots=s["slots"], **kw), s["state"]
    kw.update(initial_state=s["initial"], lengths=s["lengths"])
    out = pn.ssm_scan(s["x"], s["dt"], s["A"], s["b"], s["c"], **kw)
    if not s["train"]:
        return out
    back = pn.ssm_scan_backward(s["dy"], s["x"], s["dt"], s["A"], s["b"], s["c"], d_final_state=s["dfinal"], **kw)
    return out + (back if s["initial"] is not None else back[:8])


# ---------------------------------------------------------------- plain forms (float32)


def _silu(x):
    return x * torch.sigmoid(x)


def _silu_slope(x):
    p = torch.sigmoid(x)
    return p * (1.0 + x * (1.0 - p))


def _live(s):
    """Tokens of each sequence [B], and which rows are tokens [B, T, 1]."""
    B, T = s["B"], s["T"]
    t = torch.arange(T, device="cuda")
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device="cuda")
    return n, (t < n[:, None])[..., None]


def _conv(s):
    B, T, D, W, dt = s["B"], s["T"], s["D"], s["W"], s["x"].dtype
    n, live = _live(s)
    past = s["initial"].float() if s["initial"] is not None else torch.zeros(B, W - 1, D, device="cuda")
    x = torch.cat((past, torch.where(live, s["x"].float(), 0.0)), 1)              # [B, W - 1 + T, D]
    windows = x.unfold(1, W, 1)                                                   # [B, T, D, W]: the taps of each token
    pre = (windows * s["weight"]).sum(-1) + s["bias"]
    last = n[:, None] + torch.arange(W - 1, device="cuda")                        # rows of the final state in x
    at = last[..., None].expand(B, W - 1, D)
    out = (torch.where(live, _silu(pre), 0.0).to(dt), x.gather(1, at).to(dt))
    if not s["train"]:
        return out
    d = torch.where(live, s["dy"].float() * _silu_slope(pre), 0.0)
    dx = (torch.nn.functional.pad(d, (0, 0, W - 1, W - 1)).unfold(1, W, 1) * s["weight"].flip(1)).sum(-1)
    if s["dfinal"] is not None:
        dx = dx.scatter_add(1, at, s["dfinal"].float())
    out += (torch.where(live, dx[:, W - 1:], 0.0).to(dt), (d[..., None] * windows).sum((0, 1)), d.sum((0, 1)))
    return out if s["initial"] is None else out + (dx[:, :W - 1].to(dt),)


def _conv_step(s):
    at = s["slots"].long()
    x = torch.cat((s["state"][at], s["x"][:, None]), 1)                           # [B, W, D]
    s["state"][at] = x[:, 1:]
    return _silu((x.float() * s["weight"].T).sum(1) + s["bias"]).to(s["x"].dtype), s["state"]


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(x.clamp(max=20.0))))


def _scan_step(s):
    at, D, G = s["slots"].long(), s["D"], s["G"]
    x, b, c = s["x"].float(), s["b"].float().repeat_interleave(D // G, 1), s["c"].float().repeat_interleave(D // G, 1)
    d = _softplus(s["dt"].float() + s["dt_bias"])
    h = s["state"][at] * torch.exp(d[..., None] * s["A"]) + (d * x)[..., None] * b
    s["state"][at] = h
    return (((h * c).sum(-1) + s["skip"] * x) * _silu(s["gate"].float())).to(s["x"].dtype), s["state"]


def _join(ends, decays, first):
    """States at the start of each of K stretches from those that they leave alone, their decays and the first; and after."""
    h, starts = first, []
    for k in range(ends.shape[1]):
        starts.append(h)
        h = decays[:, k] * h + ends[:, k]
    return torch.stack(starts, 1), h


def _scan(s):
    """Stretches of about sqrt(T) tokens side by side, token by token in each: first what each leaves alone, then joined."""
    B, T, D, N, G, A, dt = s["B"], s["T"], s["D"], s["N"], s["G"], s["A"], s["x"].dtype
    _, live = _live(s)
    C = max(1, round(T ** 0.5))
    K = (T + C - 1) // C

    def rows(v):                                                                  # [B, T, ...] -> [B, K, C, ...]
        v = torch.where(live.unflatten(2, (1,) * (v.dim() - 2)), v.float(), 0.0)
        return torch.nn.functional.pad(v, (0, 0) * (v.dim() - 2) + (0, K * C - T)).unflatten(1, (K, C))

    raw = s["dt"].float() + s["dt_bias"]
    x, z, b, c, d = (rows(v) for v in (s["x"], s["gate"], s["b"], s["c"], _softplus(raw)))   # d 0: the state is kept
    u = d * x
    decay = torch.exp(d.sum(2)[..., None] * A)                                    # of a whole stretch
    wide = lambda v, i: v[:, :, i].repeat_interleave(D // G, 2)                   # noqa: E731  [B, K, D, N]
    step = lambda h, i: h * torch.exp(d[:, :, i, :, None] * A) + u[:, :, i, :, None] * wide(b, i)   # noqa: E731
    h0 = s["initial"] if s["initial"] is not None else torch.zeros(B, D, N, device="cuda")
    h = torch.zeros(B, K, D, N, device="cuda")
    if K > 1:
        for i in range(C):
            h = step(h, i)
    h, _ = _join(h, decay, h0)
    y, states = torch.empty_like(x), []
    for i in range(C):
        if s["train"]:
            states.append(h)
        h = step(h, i)
        y[:, :, i] = (h * wide(c, i)).sum(-1)
    y = y + s["skip"] * x
    back = lambda v: v.flatten(1, 2)[:, :T]                                       # noqa: E731
    out = (back(y * _silu(z)).to(dt), h[:, -1].contiguous())
    if not s["train"]:
        return out
    dy = rows(s["dy"])
    g, dz = dy * _silu(z), dy * y * _silu_slope(z)
    r = torch.zeros(B, K, D, N, device="cuda")
    pull = lambda r, i: r + g[:, :, i, :, None] * wide(c, i)                      # noqa: E731
    if K > 1:
        for i in reversed(range(C)):
            r = pull(r, i) * torch.exp(d[:, :, i, :, None] * A)
    dT = s["dfinal"] if s["dfinal"] is not None else torch.zeros(B, D, N, device="cuda")
    r, _ = _join(r.flip(1), decay.flip(1), dT)
    r = r.flip(1).contiguous()
    dx, dd, db, dc, dA = s["skip"] * g, torch.empty_like(x), torch.empty_like(b), torch.empty_like(c), torch.zeros_like(A)
    for i in reversed(range(C)):
        r = pull(r, i)                                                            # the gradient of the state after token i
        bi, a = wide(b, i), torch.exp(d[:, :, i, :, None] * A)
        kept = a * states[i]
        w = r * kept
        to_u = (r * bi).sum(-1)
        dx[:, :, i] += d[:, :, i] * to_u
        dd[:, :, i] = x[:, :, i] * to_u + (w * A).sum(-1)
        db[:, :, i] = (r * u[:, :, i, :, None]).unflatten(2, (G, D // G)).sum(3)
        dc[:, :, i] = ((kept + u[:, :, i, :, None] * bi) * g[:, :, i, :, None]).unflatten(2, (G, D // G)).sum(3)
        dA += (w * d[:, :, i, :, None]).sum((0, 1))
        r = a * r
        states[i] = None
    ddt = torch.where(live, back(dd) * torch.sigmoid(raw), 0.0)
    out += (back(dx).to(dt), ddt.to(dt), dA, back(db).to(dt), back(dc).to(dt), (g * x).sum((0, 1, 2)), back(dz).to(dt),
            ddt.sum((0, 1)))
    return out if s["initial"] is None else out + (r[:, 0].contiguous(),)




def _norm(s):
    x, r = s["x"].float(), s["r"].float()
    z = s["gate_"].float() if s["gate"] else None
    u = x if z is None else x * _silu(z)
    ru = torch.rsqrt(u.square().mean(-1, keepdim=True) + s["eps"])
    p = u * ru * s["pw"] if s["post"] else u
    t = r + (p * s["sc"] if s["scale"] else p)
    rt = torch.rsqrt(t.square().mean(-1, keepdim=True) + s["eps"])
    hat = t * rt
    out = ((hat * s["w"]).to(s["x"].dtype), t.to(s["r"].dtype))
    if not s["train"]:
        return out
    dy = s["dy"].float()
    e = dy * s["w"]
    dt = s["ds"].float() + rt * (e - hat * (e * hat).mean(-1, keepdim=True))
    dp = dt * s["sc"] if s["scale"] else dt
    du = dp
    if s["post"]:
        n, e = u * ru, dp * s["pw"]
        du = ru * (e - n * (e * n).mean(-1, keepdim=True))
    out += ((du if z is None else du * _silu(z)).to(s["x"].dtype), (dy * hat).sum((0, 1)), dt.to(s["r"].dtype))
    if z is not None:
        out += ((du * x * _silu_slope(z)).to(s["x"].dtype),)
    if s["post"]:
        out += ((dp * n).sum((0, 1)),)
    if s["scale"]:
        out += ((dt * p).sum((0, 1)),)
    return out


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    op, B, D = case["op"], case["B"], case["D"]
    F = torch.float64

    def logistic(v):
        return 1.0 / (1.0 + torch.exp(-v))

    if op == "conv_step":
        w, out = s["weight"].to(F), []
        for b, at in enumerate(s["slots"].tolist()):
            x = torch.cat((s["state"][at], s["x"][b:b + 1]))
            pre = s["bias"].to(F) + torch.einsum("kd,dk->d", x.to(F), w)
            out.append(pre * logistic(pre))
            s["state"][at] = x[1:]
        return torch.stack(out), s["state"].to(F)
    if op == "conv":
        T, W = case["T"], case["W"]
        w, bias = s["weight"].to(F), s["bias"].to(F)
        y, dx = torch.zeros(B, T, D, device="cuda", dtype=F), torch.zeros(B, T, D, device="cuda", dtype=F)
        last, d0 = (torch.zeros(B, W - 1, D, device="cuda", dtype=F) for _ in range(2))
        dw, db = torch.zeros_like(w), torch.zeros_like(bias)
        for b in range(B):
            n = int(s["lengths"][b]) if s["lengths"] is not None else T
            past = s["initial"][b].to(F) if s["initial"] is not None else torch.zeros(W - 1, D, device="cuda", dtype=F)
            x = torch.cat((past, s["x"][b, :n].to(F)))
            pre = bias + sum(w[:, k] * x[k:k + n] for k in range(W))
            p = logistic(pre)
            y[b, :n] = pre * p
            last[b] = x[n:]
            if case["train"]:
                d = s["dy"][b, :n].to(F) * p * (1.0 + pre * (1.0 - p))
                full = torch.zeros_like(x)
                for k in range(W):
                    full[k:k + n] += w[:, k] * d
                    dw[:, k] += (d * x[k:k + n]).sum(0)
                if s["dfinal"] is not None:
                    full[n:] += s["dfinal"][b].to(F)
                db += d.sum(0)
                d0[b], dx[b, :n] = full[:W - 1], full[W - 1:]
        if not case["train"]:
            return y, last
        return (y, last, dx, dw, db) + ((d0,) if s["initial"] is not None else ())
    if op == "norm":
        x, r, w = s["x"].to(F), s["r"].to(F), s["w"].to(F)
        sg = s["gate_"].to(F) if case["gate"] else None
        act = sg * logistic(sg) if case["gate"] else torch.ones((), device="cuda", dtype=F)
        scale = s["sc"].to(F) if case["scale"] else torch.ones(D, device="cuda", dtype=F)
        u = x * act
        m = (u * u).sum(-1, keepdim=True) / D + s["eps"] if case["post"] else torch.ones((), device="cuda", dtype=F)
        pw = s["pw"].to(F) if case["post"] else torch.ones(D, device="cuda", dtype=F)
        t = r + scale * pw * u / m.sqrt()
        q = (t * t).sum(-1, keepdim=True) / D + s["eps"]
        out = (w * t / q.sqrt(), t)
        if not case["train"]:
            return out
        dy = s["dy"].to(F)
        dt = s["ds"].to(F) + dy * w / q.sqrt() - t * (dy * w * t).sum(-1, keepdim=True) / (D * q ** 1.5)
        k = dt * scale * pw
        du = k / m.sqrt() - (u * (k * u).sum(-1, keepdim=True) / (D * m ** 1.5) if case["post"] else 0.0)
        out += (du * act, (dy * t / q.sqrt()).sum((0, 1)), dt)
        if case["gate"]:
            l = logistic(sg)
            out += (du * x * (l + act * (1.0 - l)),)
        if case["post"]:
            out += ((dt * scale * u / m.sqrt()).sum((0, 1)),)
        if case["scale"]:
            out += ((dt * pw * u / m.sqrt()).sum((0, 1)),)
        return out
    N, G = case["N"], case["G"]
    A, skip, bias = s["A"].to(F), s["skip"].to(F), s["dt_bias"].to(F)
    group = torch.arange(D, device="cuda") // (D // G)

    def token(x, dt, z, b, c, h):
        """One token: (y before its gate, its gate's sigmoid, step, decay, kept state, new state)."""
        v = dt.to(F) + bias
        d = torch.maximum(v, torch.zeros_like(v)) + torch.log1p(torch.exp(-v.abs()))
        a = torch.exp(d[..., None] * A)
        kept = a * h
        new = kept + (d * x.to(F))[..., None] * b.to(F)[:, group]
        return (new * c.to(F)[:, group]).sum(-1) + skip * x.to(F), logistic(z.to(F)), d, a, kept, new

    if op == "scan_step":
        at = s["slots"].long()
        y, p, _, _, _, h = token(s["x"], s["dt"], s["gate"], s["b"], s["c"], s["state"][at].to(F))
        state = s["state"].to(F)
        state[at] = h
        return y * p * s["gate"].to(F), state
    T = case["T"]
    if T * (4 if case["train"] else 1) * max(1.0, B * D * N / 1e6) > 1e5:
        return None                                     # token by token this takes too long
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device="cuda")
    h = s["initial"].to(F) if s["initial"] is not None else torch.zeros(B, D, N, device="cuda", dtype=F)
    y, keep = torch.zeros(B, T, D, device="cuda", dtype=F), []
    for t in range(T):
        on = (t < n)[:, None, None]
        yt, p, _, _, _, new = token(*(s[k][:, t] for k in ("x", "dt", "gate", "b", "c")), h)
        y[:, t] = yt * p * s["gate"][:, t].to(F) * on[..., 0]
        if case["train"]:
            keep.append(h)
        h = torch.where(on, new, h)
    if not case["train"]:
        return y, h
    z64 = lambda *shape: torch.zeros(*shape, device="cuda", dtype=F)              # noqa: E731
    dx, ddt, dz, db, dc = z64(B, T, D), z64(B, T, D), z64(B, T, D), z64(B, T, G, N), z64(B, T, G, N)
    dA, dskip = torch.zeros_like(A), torch.zeros_like(skip)
    R = s["dfinal"].to(F) if s["dfinal"] is not None else z64(B, D, N)            # gradient of the state after a token
    for t in reversed(range(T)):
        on = (t < n)[:, None, None].to(F)
        x, dt, z, b, c = (s[k][:, t] for k in ("x", "dt", "gate", "b", "c"))
        yt, p, d, a, kept, new = token(x, dt, z, b, c, keep[t])
        x, z, dyt, bt, ct = x.to(F), z.to(F), s["dy"][:, t].to(F) * on[..., 0], b.to(F)[:, group], c.to(F)[:, group]
        g = dyt * z * p
        dz[:, t] = dyt * yt * (p + z * p * (1.0 - p))
        R = R + g[..., None] * ct
        live = R * on
        du = (live * bt).sum(-1)
        dd = du * x + (live * kept * A).sum(-1)
        dx[:, t] = du * d + skip * g
        ddt[:, t] = dd * logistic(dt.to(F) + bias)
        db[:, t].index_add_(1, group, live * (d * x)[..., None])
        dc[:, t].index_add_(1, group, g[..., None] * new)
        dA += (live * kept * d[..., None]).sum(0)
        dskip += (g * x).sum(0)
        R = torch.where(on > 0, a * R, R)
        keep[t] = None
    out = (y, h, dx, ddt, dA, db, dc, dskip, dz, ddt.sum((0, 1)))
    return out if s["initial"] is None else out + (R,)
