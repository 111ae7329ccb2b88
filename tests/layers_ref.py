"""Plain 64-bit references of the layer operators, step by step from their definitions, and the
gradients by the chain rule; torch on the CPU, nothing shared with the kernels."""

import math

import torch


def softplus(v):
    return torch.logaddexp(v, torch.zeros_like(v))


def gated_scan(x, r, i, lam, c=8.0, h0=None, reset=None):
    """(y, last) of the gated recurrence in float64, one step after another."""
    x, r, i, lam = (t.double() for t in (x, r, i, lam))
    B, L, D = x.shape
    h = torch.zeros(B, D, dtype=torch.float64) if h0 is None else h0.double()
    ys = []
    for t in range(L):
        s = c * softplus(lam) * torch.sigmoid(r[:, t])
        a, m = torch.exp(-s), torch.sqrt(-torch.expm1(-2 * s))
        if reset is not None:
            on = reset[:, t, None].bool()
            a = torch.where(on, torch.zeros_like(a), a)
            m = torch.where(on, torch.ones_like(m), m)
        h = a * h + m * torch.sigmoid(i[:, t]) * x[:, t]
        ys.append(h)
    y = torch.stack(ys, 1) if L else torch.zeros(B, 0, D, dtype=torch.float64)
    return y, h


def gated_scan_bwd(x, r, i, lam, dy, c=8.0, h0=None, reset=None, dlast=None):
    """Gradients by the chain rule, from the last step to the first."""
    y, _ = gated_scan(x, r, i, lam, c, h0, reset)
    x, r, i, lam, dy = (t.double() for t in (x, r, i, lam, dy))
    B, L, D = x.shape
    zero = torch.zeros(B, D, dtype=torch.float64)
    start = zero if h0 is None else h0.double()
    mu = zero if dlast is None else dlast.double()
    dx, dr, di = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
    dlam = torch.zeros(D, dtype=torch.float64)
    for t in range(L - 1, -1, -1):
        sr, si = torch.sigmoid(r[:, t]), torch.sigmoid(i[:, t])
        s = c * softplus(lam) * sr
        a, m = torch.exp(-s), torch.sqrt(-torch.expm1(-2 * s))
        # dm/ds = e^{-2s} / m, and m ~ sqrt(2s) at s = 0, where s dm/ds vanishes
        sdm = torch.where(s > 0, s * torch.exp(-2 * s) / torch.where(m > 0, m, torch.ones_like(m)), torch.zeros_like(s))
        sda = -s * a
        if reset is not None:
            on = reset[:, t, None].bool()
            a, m = torch.where(on, zero, a), torch.where(on, torch.ones_like(m), m)
            sda, sdm = torch.where(on, zero, sda), torch.where(on, zero, sdm)
        g = dy[:, t] + mu
        before = y[:, t - 1] if t else start
        q = g * (sda * before + sdm * si * x[:, t])
        dx[:, t] = g * m * si
        di[:, t] = g * m * x[:, t] * si * (1 - si)
        dr[:, t] = q * (1 - sr)
        dlam += (q * torch.sigmoid(lam) / softplus(lam)).sum(0)
        mu = g * a
    return {"x": dx, "r": dr, "i": di, "lam": dlam, "h0": mu}


def layer_norm(t, weight=None, bias=None, eps=1e-5):
    t = t.double()
    mean = t.mean(-1, keepdim=True)
    y = (t - mean) / torch.sqrt((t - mean).square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    return y if bias is None else y + bias.double()


def layer_norm_bwd(t, weight, dy, eps=1e-5, dresidual=None):
    t, dy = t.double(), dy.double()
    mean = t.mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt((t - mean).square().mean(-1, keepdim=True) + eps)
    n = (t - mean) * rstd
    g = dy if weight is None else dy * weight.double()
    dx = rstd * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    if dresidual is not None:
        dx = dx + dresidual.double()
    rows = tuple(range(t.dim() - 1))
    return {"x": dx, "weight": (dy * n).sum(rows), "bias": dy.sum(rows)}


def embedding(ids, weight, scale=1.0):
    V = weight.shape[0]
    ok = (ids >= 0) & (ids < V)
    if V == 0:
        return torch.zeros(*ids.shape, weight.shape[1], dtype=torch.float64)
    y = weight.double()[ids.clamp(0, V - 1).long()] * scale
    return torch.where(ok[..., None], y, torch.zeros_like(y))


def embedding_bwd(ids, dy, vocab, scale=1.0):
    dw = torch.zeros(vocab, dy.shape[-1], dtype=torch.float64)
    flat, rows = ids.reshape(-1).tolist(), dy.double().reshape(ids.numel(), dy.shape[-1])
    for t, v in enumerate(flat):
        if 0 <= v < vocab:
            dw[v] += rows[t] * scale
    return dw


def lam_for(decays, c=8.0):
    """lam whose decay with an open gate is the given one."""
    return torch.log(torch.expm1(-torch.log(decays.double()) / c)).float()


def act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    k = math.sqrt(2 / math.pi)
    return 0.5 * g * (1 + torch.tanh(k * (g + 0.044715 * g ** 3)))


def dact(g, kind):
    if kind == "silu":
        s = torch.sigmoid(g)
        return s * (1 + g * (1 - s))
    k = math.sqrt(2 / math.pi)
    th = torch.tanh(k * (g + 0.044715 * g ** 3))
    return 0.5 * (1 + th) + 0.5 * g * (1 - th * th) * k * (1 + 3 * 0.044715 * g * g)


def gated_ffn(x, wg, wu, kind="silu"):
    x, wg, wu = x.double(), wg.double(), wu.double()
    return act(x @ wg.t(), kind) * (x @ wu.t())


def gated_ffn_bwd(x, wg, wu, dh, kind="silu"):
    x, wg, wu, dh = x.double(), wg.double(), wu.double(), dh.double()
    g, u = x @ wg.t(), x @ wu.t()
    dg, du = dh * u * dact(g, kind), dh * act(g, kind)
    return {"x": dg @ wg + du @ wu, "w_gate": dg.t() @ x, "w_up": du.t() @ x}
