"""The layer operators around the scan, as they are measured: the gated linear recurrence, layer
norm with its residual, the token embedding and the gated feed-forward block, each with its
gradient. ``run`` computes a case either in plain torch operations (fp32, rounded once at the end)
or, where ``own`` is set, through ``selective_state_space_29_amd.layers``.

Definitions (s = softplus, sg = logistic sigmoid; statistics, states and sums in fp32 or more):

* gated scan, x, r, i (batch, len, dim), lam (dim):
  log a = -c s(lam) sg(r), 0 decay where reset is set;  b = sqrt(1 - a^2) sg(i) x;
  h_t = a_t h_{t-1} + b_t;  y = h in x's dtype, last_state = h of the last step in fp32.
* layer norm with residual: t = x + residual rounded to x's dtype (t = x without one),
  y = (t - mean) / sqrt(var + eps) * weight + bias; backward adds the gradient that reaches t.
* embedding: y = scale * weight[id], zeros for an id outside [0, vocab); the gradient sums the rows
  of each id.
* gated feed-forward: h = silu(x Wg^T) * (x Wu^T).

Activations' gradients come in the activations' dtype, parameters' gradients in the parameters'.
"""

import math

import torch

own = False

C = 8.0      # the recurrence's gate constant
EPS = 1e-5   # layer norm
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one decode step of 32 streams at the width of the Mamba-130m layer: a call's latency
        dict(name="scan_step", op="scan", train=False, dtype="bf16", batch=32, len=1, dim=1536, h0=True, reset=False, merged=False),
        # prompt processing at the Mamba-130m layer's shape, final state kept for decoding
        dict(name="scan_fwd", op="scan", train=False, dtype="bf16", batch=8, len=2048, dim=1536, h0=False, reset=False, merged=False),
        # a long genomic stretch, sequences of many lengths packed one after another
        dict(name="scan_long", op="scan", train=False, dtype="bf16", batch=4, len=100000, dim=1024, h0=False, reset=True, merged=False),
        # a training step of the recurrence; x and the gates are slices of one projection's output
        dict(name="scan_train", op="scan", train=True, dtype="bf16", batch=8, len=2048, dim=1536, h0=False, reset=False, merged=True),
        # the same in fp32, odd in every size, from a given state, with packed sequences
        dict(name="scan_train_odd", op="scan", train=True, dtype="f32", batch=3, len=2777, dim=1001, h0=True, reset=True, merged=False),
        # pre-norm of a block: the residual added on the way
        dict(name="norm_fwd", op="norm", train=False, dtype="bf16", rows=16384, dim=768, residual=True),
        # the norm of a wider model in training, with the residual stream's own gradient
        dict(name="norm_train", op="norm", train=True, dtype="bf16", rows=16384, dim=2048, residual=True),
        # fp32, odd sizes, no residual
        dict(name="norm_train_odd", op="norm", train=True, dtype="f32", rows=5003, dim=1001, residual=False),
        # the embedding of a training batch, padded at the end of each sequence
        dict(name="embed_fwd", op="embed", train=False, dtype="bf16", batch=8, len=2048, vocab=50000, dim=768, pad=True),
        # its gradient: word frequencies fall as 1/rank, so few ids take many tokens and most ids none
        dict(name="embed_bwd", op="embed", train=True, dtype="bf16", batch=8, len=2048, vocab=50000, dim=768, pad=True),
        # one decode step of eight streams through the feed-forward block: the weights are read once
        dict(name="ffn_step", op="ffn", train=False, dtype="bf16", rows=8, dim=2048, hidden=8192),
        # a training step of the feed-forward block over a batch of 8 x 2048 tokens
        dict(name="ffn_train", op="ffn", train=True, dtype="bf16", rows=16384, dim=768, hidden=2048),
    ]


def _spread(rng, lo, hi):
    """A size spread over [lo, hi], over its logarithm where that is wide; odd ones as they fall."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))) if hi > 10 * lo else rng.randint(lo, hi)
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["scan", "scan", "norm", "embed", "ffn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.5
    if op == "scan":
        dim, batch = _spread(rng, 64, 4096), rng.randint(1, 32)
        most = (25_000_000 if train else 50_000_000) // (dim * batch)
        length = 1 if rng.random() < 0.2 else max(1, min(100000, _spread(rng, 2, max(3, most))))
        return dict(op=op, train=train, dtype=dtype, batch=batch, len=length, dim=dim, h0=rng.random() < 0.5,
                    reset=rng.random() < 0.5, merged=rng.random() < 0.5 and 3 * dim != 3072)
    if op == "norm":
        dim = _spread(rng, 64, 8192)
        return dict(op=op, train=train, dtype=dtype, rows=_spread(rng, 1, max(2, 33_000_000 // dim)), dim=dim,
                    residual=rng.random() < 0.5)
    if op == "embed":
        dim, vocab = _spread(rng, 64, 2048), _spread(rng, 200, 50000)
        return dict(op=op, train=train, dtype=dtype, batch=rng.randint(1, 8), len=_spread(rng, 1, 4096), vocab=vocab,
                    dim=min(dim, 38_000_000 // vocab), pad=rng.random() < 0.5)
    dim, hidden = _spread(rng, 128, 2048), _spread(rng, 128, 8192)
    most = max(2, min(16384, 25_000_000_000 // (dim * hidden)))
    rows = rng.randint(1, 16) if rng.random() < 0.4 else _spread(rng, 1, most)
    return dict(op=op, train=train, dtype="bf16", rows=rows, dim=dim, hidden=hidden)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = DT[case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)

    s = dict(case)
    if case["op"] == "scan":
        B, L, D = case["batch"], case["len"], case["dim"]
        if case["merged"]:
            p = normal(B, L, 3 * D)
            s["x"], s["r"], s["i"] = p[..., :D], p[..., D:2 * D], p[..., 2 * D:]
        else:
            s["x"], s["r"], s["i"] = normal(B, L, D), normal(B, L, D), normal(B, L, D)
        # decays between 0.9 and 0.999 a step where the gate is fully open
        decay = 0.9 + 0.099 * torch.rand(D, generator=g, device=DEV, dtype=torch.float64)
        s["lam"] = torch.log(torch.expm1(-torch.log(decay) / C)).float()
        s["h0v"] = normal(B, D, dtype=torch.float32) if case["h0"] else None
        # sequences of 700 steps at the mean; without a state to go on from, every row begins one
        s["resetv"] = None
        if case["reset"]:
            s["resetv"] = torch.rand(B, L, generator=g, device=DEV) < 1 / 700
            s["resetv"][:, 0] |= not case["h0"]
        if case["train"]:
            s["dy"] = normal(B, L, D)
            s["dlast"] = normal(B, D, dtype=torch.float32)
    elif case["op"] == "norm":
        M, D = case["rows"], case["dim"]
        s["x"] = normal(M, D)
        s["res"] = normal(M, D, std=2.0) if case["residual"] else None
        s["w"] = 1 + normal(D, std=0.1, dtype=torch.float32)
        s["b"] = normal(D, std=0.1, dtype=torch.float32)
        if case["train"]:
            s["dy"] = normal(M, D)
            s["dres"] = normal(M, D) if case["residual"] else None
    elif case["op"] == "embed":
        B, L, V, D = case["batch"], case["len"], case["vocab"], case["dim"]
        u = torch.rand(B, L, generator=g, device=DEV, dtype=torch.float64)
        ids = (torch.pow(float(V + 1), u).long() - 1).clamp_(0, V - 1)  # P(rank) ~ 1 / rank
        if case["pad"]:
            n = torch.randint(L // 2, L + 1, (B, 1), generator=g, device=DEV)
            ids = torch.where(torch.arange(L, device=DEV)[None] < n, ids, -1)
        s["ids"] = ids
        s["scale"] = math.sqrt(D)
        if case["train"]:
            s["dy"] = normal(B, L, D)
        else:
            s["w"] = normal(V, D, std=D ** -0.5)
    else:
        M, K, F = case["rows"], case["dim"], case["hidden"]
        s["x"] = normal(M, K)
        s["wg"] = normal(F, K, std=K ** -0.5)
        s["wu"] = normal(F, K, std=K ** -0.5)
        if case["train"]:
            s["dh"] = normal(M, F)
    return s


# ---- the framework's operators ----

def _run_own(s):
    from selective_state_space_29_amd import layers

    if s["op"] == "scan":
        kw = dict(c=C, h0=s["h0v"], reset=s["resetv"])
        if not s["train"]:
            return layers.gated_scan_fn(s["x"], s["r"], s["i"], s["lam"], return_last_state=True, **kw)
        ck = torch.empty(layers.gated_checkpoint_shape(*s["x"].shape), dtype=torch.float32, device=s["x"].device)
        y, last = layers.gated_scan_fn(s["x"], s["r"], s["i"], s["lam"], return_last_state=True, checkpoints_out=ck, **kw)
        g = layers.gated_scan_bwd(s["x"], s["r"], s["i"], s["lam"], s["dy"], dlast_state=s["dlast"], checkpoints=ck, **kw)
        return (y, last, g["x"], g["r"], g["i"], g["lam"]) + ((g["h0"],) if s["h0"] else ())
    if s["op"] == "norm":
        if not s["train"]:
            return layers.layer_norm_fn(s["x"], s["w"], s["b"], EPS, residual=s["res"])
        out, stats = layers.layer_norm_fn(s["x"], s["w"], s["b"], EPS, residual=s["res"], return_stats=True)
        t = out[1] if s["residual"] else s["x"]
        g = layers.layer_norm_bwd(t, s["w"], s["dy"], stats, dresidual=s["dres"])
        return (*(out if s["residual"] else (out,)), g["x"], g["weight"], g["bias"])
    if s["op"] == "embed":
        if not s["train"]:
            return layers.embedding_fn(s["ids"], s["w"], scale=s["scale"])
        return layers.embedding_bwd(s["ids"], s["dy"], s["vocab"], scale=s["scale"])
    h = layers.gated_ffn_fn(s["x"], s["wg"], s["wu"])
    if not s["train"]:
        return h
    g = layers.gated_ffn_bwd(s["x"], s["wg"], s["wu"], s["dh"])
    return h, g["x"], g["w_gate"], g["w_up"]


# ---- the plain forms, in fp32 ----

def _doubling(a, h):
    """All h_t = a_t h_{t-1} + b_t at once (h holds the b_t), along dimension 1: pairs of steps are
    combined over distances 1, 2, 4, ..."""
    n = 1
    while n < h.shape[1]:
        h = torch.cat([h[:, :n], h[:, n:] + a[:, n:] * h[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return h


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-torch.abs(v)))


def _run_scan(s):
    dt = s["x"].dtype
    x, r, i, lam = s["x"].float(), s["r"].float(), s["i"].float(), s["lam"]
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    v = (C * _softplus(lam)) * sr                     # -log a
    keep = None if s["resetv"] is None else (~s["resetv"]).float()[..., None]
    a = torch.exp(-v)
    e = -torch.expm1(-2 * v)                          # 1 - a^2
    if keep is not None:
        a, e = a * keep, torch.where(keep > 0, e, 1.0)
    m = torch.sqrt(e)
    b = m * si * x
    if s["h0v"] is not None:
        b[:, 0] += a[:, 0] * s["h0v"]
    h = _doubling(a, b)
    y, last = h.to(dt), h[:, -1].clone()
    if not s["train"]:
        return y, last
    # backward: G_t = dy_t + a_{t+1} G_{t+1}, the recurrence run from the end
    dy = s["dy"].float().clone()
    dy[:, -1] += s["dlast"]
    nxt = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    G = _doubling(nxt.flip(1), dy.flip(1)).flip(1)
    first = torch.zeros_like(h[:, :1]) if s["h0v"] is None else s["h0v"][:, None]
    prev = torch.cat([first, h[:, :-1]], 1)
    q = G * (a * a * si * x * (v / m) - a * v * prev)  # v dLoss/dv; a = 0 after a reset
    dx = G * m * si
    di = G * m * x * si * (1 - si)
    dr = q * (1 - sr)
    dlam = q.sum((0, 1)) * torch.sigmoid(lam) / _softplus(lam)
    out = (y, last, dx.to(dt), dr.to(dt), di.to(dt), dlam)
    return out + ((G[:, 0] * a[:, 0],) if s["h0"] else ())


def _run_norm(s):
    dt = s["x"].dtype
    t = s["x"].float()
    if s["res"] is not None:
        t = (t + s["res"].float()).to(dt).float()
    mean = t.mean(-1, keepdim=True)
    rstd = torch.rsqrt((t - mean).square().mean(-1, keepdim=True) + EPS)
    xh = (t - mean) * rstd
    y = (xh * s["w"] + s["b"]).to(dt)
    out = (y,) if s["res"] is None else (y, t.to(dt))
    if not s["train"]:
        return out if s["res"] is not None else y
    dy = s["dy"].float()
    g = dy * s["w"]
    dx = rstd * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    return (*out, dx.to(dt), (dy * xh).sum(0), dy.sum(0))


def _run_embed(s):
    ids, V = s["ids"].reshape(-1), s["vocab"]
    ok = ((ids >= 0) & (ids < V))[:, None]
    at = ids.clamp(0, V - 1)
    if not s["train"]:
        y = torch.where(ok, s["w"][at].float() * s["scale"], 0.0)
        return y.to(s["w"].dtype).reshape(*s["ids"].shape, -1)
    dy = s["dy"].reshape(-1, s["dy"].shape[-1])
    dw = torch.zeros(V, dy.shape[1], device=dy.device)
    dw.index_add_(0, at, torch.where(ok, dy.float(), 0.0))
    return (dw * s["scale"]).to(dy.dtype)


def _run_ffn(s):
    dt = s["x"].dtype
    x, wg, wu = s["x"].float(), s["wg"].float(), s["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    sg = torch.sigmoid(g)
    h = (g * sg * u).to(dt)
    if not s["train"]:
        return h
    dh = s["dh"].float()
    dg = dh * u * sg * (1 + g * (1 - sg))
    du = dh * g * sg
    return h, (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt)


def run(state):
    if own:
        return _run_own(state)
    return {"scan": _run_scan, "norm": _run_norm, "embed": _run_embed, "ffn": _run_ffn}[state["op"]](state)


# ---- what a pass cannot do without ----

def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "scan":
        n, rows = case["batch"] * case["len"] * case["dim"], case["batch"] * case["dim"]
        # x, r, i read, y written; training reads them and dy once more and writes three gradients
        by = 4 * n * es + rows * 4 * (1 + case["h0"]) + case["dim"] * 4
        by += case["batch"] * case["len"] if case["reset"] else 0
        if case["train"]:
            by += 4 * n * es + rows * 4 * (1 + case["h0"]) + case["dim"] * 4  # dy, dx, dr, di, dlast, dh0, dlam
        return {"bytes": by, "flops": n * (46 if case["train"] else 18)}
    if case["op"] == "norm":
        n = case["rows"] * case["dim"]
        by = 2 * n * es + case["dim"] * 8 + (2 * n * es if case["residual"] else 0)
        if case["train"]:  # dy and dx, the residual stream's gradient, dw, db
            by += 2 * n * es + (n * es if case["residual"] else 0) + case["dim"] * 8
        return {"bytes": by, "flops": n * (24 if case["train"] else 9)}
    if case["op"] == "embed":
        T, V, D = case["batch"] * case["len"], case["vocab"], case["dim"]
        if case["train"]:
            return {"bytes": T * D * es + T * 8 + V * D * es, "flops": T * D + V * D}
        return {"bytes": T * D * es + min(T, V) * D * es + T * 8, "flops": T * D}
    M, K, F = case["rows"], case["dim"], case["hidden"]
    by = (M * K + 2 * F * K + M * F) * es
    fl = 4 * M * K * F
    if case["train"]:
        by += (M * F + M * K + 2 * F * K) * es
        fl *= 3
    return {"bytes": by, "flops": fl}


# ---- the definitions in 64 bits ----

def _exact_scan(s):
    x, r, i, lam = (s[k].double() for k in ("x", "r", "i", "lam"))
    B, L, D = x.shape
    sr, si = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-i))
    loga = -C * torch.logaddexp(lam, torch.zeros_like(lam)) * sr
    a, m = torch.exp(loga), torch.sqrt(-torch.expm1(2 * loga))
    if s["resetv"] is not None:
        a.masked_fill_(s["resetv"][..., None], 0.0)
        m.masked_fill_(s["resetv"][..., None], 1.0)
    h = m * si * x
    if not s["train"]:
        del r, i, sr, si, loga, m, x
    now = torch.zeros(B, D, device=h.device, dtype=torch.float64) if s["h0v"] is None else s["h0v"].double()
    start = now
    for t in range(L):
        now = torch.addcmul(h[:, t], a[:, t], now)
        h[:, t] = now
    if not s["train"]:
        return h, now
    dx, dr, di = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    dloga = torch.empty_like(x)
    dy, G = s["dy"].double(), s["dlast"].double()
    for t in range(L - 1, -1, -1):
        G = G + dy[:, t]
        before = h[:, t - 1] if t else start
        da = G * before - G * (a[:, t] / m[:, t]) * si[:, t] * x[:, t]  # through a, and through m = sqrt(1 - a^2)
        dloga[:, t] = da * a[:, t]
        dx[:, t] = G * m[:, t] * si[:, t]
        di[:, t] = G * m[:, t] * x[:, t] * si[:, t] * (1 - si[:, t])
        G = G * a[:, t]
    dr = dloga * loga * (1 - sr)
    dlam = (dloga * (-C) * sr).sum((0, 1)) / (1 + torch.exp(-lam))
    return (h, now, dx, dr, di, dlam) + ((G,) if s["h0"] else ())


def _exact_norm(s):
    t = s["x"].double()
    if s["res"] is not None:
        t = (t + s["res"].double()).to(s["x"].dtype).double()
    D = t.shape[-1]
    c = t - t.sum(-1, keepdim=True) / D
    sd = torch.sqrt(c.square().sum(-1, keepdim=True) / D + EPS)
    w = s["w"].double()
    y = c / sd * w + s["b"].double()
    out = (y,) if s["res"] is None else (y, t)
    if not s["train"]:
        return out if s["res"] is not None else y
    dy = s["dy"].double()
    # d/dt of c/sd: the projection off the constant vector and off c
    gw = dy * w / sd
    dx = gw - gw.sum(-1, keepdim=True) / D - c * (gw * c).sum(-1, keepdim=True) / (D * sd * sd)
    if s["dres"] is not None:
        dx = dx + s["dres"].double()
    return (*out, dx, (dy * c / sd).sum(0), dy.sum(0))


def _exact_embed(s):
    ids, V = s["ids"].reshape(-1), s["vocab"]
    ok = ((ids >= 0) & (ids < V)).nonzero().reshape(-1)
    if not s["train"]:
        y = torch.zeros(ids.numel(), s["w"].shape[1], device=ids.device, dtype=torch.float64)
        y[ok] = s["w"].double()[ids[ok]] * s["scale"]
        return y.reshape(*s["ids"].shape, -1)
    dy = s["dy"].reshape(ids.numel(), -1).double()
    dw = torch.zeros(V, dy.shape[1], device=ids.device, dtype=torch.float64)
    dw.index_put_((ids[ok],), dy[ok] * s["scale"], accumulate=True)
    return dw


def _exact_ffn(s):
    x, wg, wu = s["x"].double(), s["wg"].double(), s["wu"].double()
    g, u = torch.mm(x, wg.t()), torch.mm(x, wu.t())
    act = g / (1 + torch.exp(-g))
    if not s["train"]:
        return act * u
    dh = s["dh"].double()
    slope = torch.exp(-g) / (1 + torch.exp(-g)).square() * g + 1 / (1 + torch.exp(-g))
    dg, du = dh * u * slope, dh * act
    return act * u, torch.mm(dg, wg) + torch.mm(du, wu), torch.mm(dg.t(), x), torch.mm(du.t(), x)


def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "norm": _exact_norm, "embed": _exact_embed, "ffn": _exact_ffn}[case["op"]](s)
