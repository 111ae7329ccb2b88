"""Plain 64-bit references of the block operators, step by step from their definitions, and their gradients by
the chain rule; torch on the CPU, nothing shared with the kernels."""

import torch

from layers_ref import softplus


def silu(v):
    return v * torch.sigmoid(v)


def dsilu(v):
    s = torch.sigmoid(v)
    return s * (1 + v * (1 - s))


def _seen(x, state, reset, width):
    """For each step the width values it sees, oldest first, as places in the line state + x (-1: none), and the
    places that the state after the last step holds."""
    B, L, _ = x.shape
    places, left = [], []
    for b in range(B):
        begin, rows = 0, []
        for t in range(L):
            if reset is not None and reset[b, t]:
                begin = t + width - 1
            rows.append([p if p >= begin else -1 for p in range(t, t + width)])
        places.append(rows)
        left.append([p if p >= begin else -1 for p in range(L, L + width - 1)])
    return places, left


def causal_conv(x, weight, bias=None, state=None, reset=None, activation="silu", dy=None, dlast=None):
    """(y, last state), and with dy the gradients as a dict."""
    x, weight = x.double(), weight.double()
    B, L, D = x.shape
    W = weight.shape[1]
    line = torch.cat([torch.zeros(B, W - 1, D, dtype=torch.float64) if state is None else state.double(), x], 1)
    places, left = _seen(x, state, reset, W)
    pre = torch.zeros(B, L, D, dtype=torch.float64) if bias is None else bias.double().expand(B, L, D).clone()
    last = torch.zeros(B, W - 1, D, dtype=torch.float64)
    for b in range(B):
        for t in range(L):
            for k, p in enumerate(places[b][t]):
                if p >= 0:
                    pre[b, t] += weight[:, k] * line[b, p]
        for j, p in enumerate(left[b]):
            if p >= 0:
                last[b, j] = line[b, p]
    y = silu(pre) if activation == "silu" else pre
    if dy is None:
        return y, last
    dpre = dy.double() * (dsilu(pre) if activation == "silu" else 1.0)
    dline, dw = torch.zeros_like(line), torch.zeros_like(weight)
    for b in range(B):
        for t in range(L):
            for k, p in enumerate(places[b][t]):
                if p >= 0:
                    dline[b, p] += weight[:, k] * dpre[b, t]
                    dw[:, k] += dpre[b, t] * line[b, p]
        if dlast is not None:
            for j, p in enumerate(left[b]):
                if p >= 0:
                    dline[b, p] += dlast.double()[b, j]
    return y, last, {"x": dline[:, W - 1:], "initial_state": dline[:, :W - 1], "weight": dw, "bias": dpre.sum((0, 1))}


def block_step(x, conv_state, ssm_state, conv_w, conv_b, w_x, w_dt, dt_bias, A, D=None, z=None):
    """(y, conv state, scan state) after one token."""
    x, conv_state, h, conv_w, w_x, w_dt, A = (t.double() for t in (x, conv_state, ssm_state, conv_w, w_x, w_dt, A))
    line = torch.cat([conv_state, x[:, None]], 1)
    pre = (line * conv_w.t()).sum(1)
    u = silu(pre if conv_b is None else pre + conv_b.double())
    R, N = w_dt.shape[1], A.shape[1]
    dbc = u @ w_x.t()
    delta = dbc[:, :R] @ w_dt.t()
    s = softplus(delta if dt_bias is None else delta + dt_bias.double())[..., None]
    h = torch.exp(s * A) * h + s * u[..., None] * dbc[:, None, R:R + N]
    y = (h * dbc[:, None, R + N:]).sum(-1)
    if D is not None:
        y = y + D.double() * u
    return (y if z is None else y * silu(z.double())), line[:, 1:], h


def rms_norm(t, weight=None, eps=1e-5, dy=None, dsum=None):
    """y of t, or with dy the gradients at t and in the weight."""
    t = t.double()
    rstd = 1 / torch.sqrt(t.square().mean(-1, keepdim=True) + eps)
    w = torch.ones(t.shape[-1], dtype=torch.float64) if weight is None else weight.double()
    if dy is None:
        return t * rstd * w
    n, g = t * rstd, dy.double() * w
    dt = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    if dsum is not None:
        dt = dt + dsum.double()
    return {"t": dt, "weight": (dy.double() * n).sum(tuple(range(t.dim() - 1)))}


def gated_rms_norm(x, z, weight=None, eps=1e-5, groups=1, gate_first=True, dy=None):
    """y, or with dy the gradients; a group at a time."""
    x, z = x.double(), z.double()
    D = x.shape[-1]
    w = torch.ones(D, dtype=torch.float64) if weight is None else weight.double()
    y, dx, dz, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x), torch.zeros(D, dtype=torch.float64)
    size = D // groups
    for k in range(groups):
        c = slice(k * size, (k + 1) * size)
        gate = silu(z[..., c])
        v = x[..., c] * gate if gate_first else x[..., c]
        after = torch.ones_like(gate) if gate_first else gate
        y[..., c] = rms_norm(v, w[c], eps) * after
        if dy is not None:
            d = dy.double()[..., c]
            g = rms_norm(v, w[c], eps, dy=d * after)
            dw[c] = g["weight"]
            if gate_first:
                dx[..., c], dz[..., c] = g["t"] * gate, g["t"] * x[..., c] * dsilu(z[..., c])
            else:
                dx[..., c], dz[..., c] = g["t"], d * rms_norm(v, w[c], eps) * dsilu(z[..., c])
    return y if dy is None else {"x": dx, "z": dz, "weight": dw}


def linear_cross_entropy(x, weight, target, scale=1.0, dloss=None, dlse=None):
    """(loss, lse) of rows, and with dloss or dlse the gradients as a dict."""
    x, weight = x.double(), weight.double()
    V = weight.shape[0]
    logits = scale * (x @ weight.t())
    lse = torch.logsumexp(logits, -1)
    hit = (target >= 0) & (target < V)
    at = target.long().clamp(0, V - 1)
    loss = torch.where(hit, lse - logits.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    if dloss is None and dlse is None:
        return loss, lse
    a = torch.where(hit, torch.zeros_like(lse) if dloss is None else dloss.double(), torch.zeros_like(lse))
    f = a if dlse is None else a + dlse.double()
    d = f[:, None] * torch.exp(logits - lse[:, None])
    d[torch.arange(len(at)), at] -= a
    on = ((a != 0) | (f != 0))[:, None]
    d = torch.where(on, d, torch.zeros_like(d))
    return loss, lse, {"x": scale * d @ weight, "weight": scale * d.t() @ torch.where(on, x, torch.zeros_like(x))}
