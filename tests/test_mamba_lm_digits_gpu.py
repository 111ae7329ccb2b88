"""The Mamba language model of the examples against itself in 64 bits: what its kernels lose is no more than what rounding
to bf16 loses.

Bar. The same model from elementary torch operations in fp32, rounded to bf16 where the kernels round, is another way to
round the same graph, and its distance from 64 bits says what those roundings cost. Two ways of rounding differ by chance
and not in size: the kernels' distance is at most twice the plain one's, for every parameter and for the tokens' losses, and
half a step of bf16 (2^-9 of the gradient) for the gradient's own last rounding.
"""

import copy
import types

import pytest
import torch
import torch.nn.functional as F

import test_mamba_lm_gpu as lm

pytestmark = pytest.mark.gpu


class Exact:
    """The block operators in the inputs' own precision."""

    @staticmethod
    def rms_norm(x, w, residual=None, scale=1.0):
        t = x if residual is None else residual + scale * x
        y = t / torch.sqrt(t.square().mean(-1, keepdim=True) + 1e-5) * w
        return y if residual is None else (y, t)

    @staticmethod
    def gated_rms_norm(x, z, w):
        return Exact.rms_norm(x * F.silu(z), w)

    @staticmethod
    def causal_conv(x, w, b, scan_layout):
        p = F.pad(x, (0, 0, 3, 0))
        return F.silu(sum(p[:, k:k + x.shape[1]] * w[:, 0, k] for k in range(4)) + b)


def embedding(ids, weight, scale):
    return torch.where((ids >= 0)[..., None], weight[ids.clamp(min=0)] * scale, torch.zeros((), dtype=weight.dtype, device=weight.device))


def selective_scan(u, delta, A, B, C, D, delta_bias, delta_softplus):
    s = F.softplus(delta + delta_bias[:, None])
    h, out = torch.zeros(*u.shape[:2], A.shape[1], dtype=u.dtype, device=u.device), []
    for t in range(u.shape[2]):
        h = torch.exp(s[:, :, t, None] * A) * h + (s[:, :, t] * u[:, :, t])[..., None] * B[:, None, :, t]
        out.append((h * C[:, None, :, t]).sum(-1) + D * u[:, :, t])
    return torch.stack(out, 2)


def gradients(model, ids, target, losses):
    """The tokens' losses and, of their mean, every parameter's gradient."""
    model.zero_grad()
    each = losses(model.hidden(ids), model.embed, target)
    (each.sum() / ((target >= 0) & (target < 50)).sum()).backward()
    return {"losses": each.detach(), **{n: p.grad.clone() for n, p in model.named_parameters()}}


def plain_losses(x, w, target):
    up = torch.float64 if x.dtype == torch.float64 else torch.float32
    return F.cross_entropy(x.flatten(0, 1).to(up) @ w.to(up).t(), target.flatten(), ignore_index=-100, reduction="none").view(target.shape)


def test_gradients_lose_no_more_than_rounding():
    ex = lm.example()
    model = lm.small_model(ex)
    ids, target = ex.sequences(3, 90, 50, "cuda", torch.Generator().manual_seed(2))
    got = gradients(model, ids, target, lambda x, w, t: ex.block.linear_cross_entropy(x, w, t, reduction="none"))
    ex.block = lm.Plain
    plain = gradients(model, ids, target, plain_losses)
    ex.block, ex.layers, ex.scan = Exact, types.SimpleNamespace(embedding=embedding), types.SimpleNamespace(selective_scan=selective_scan)
    exact = gradients(copy.deepcopy(model).double(), ids, target, plain_losses)
    assert len(exact) == 1 + len(list(model.parameters()))
    for n, want in exact.items():
        far, allowed = (float((v[n].double() - want).norm()) for v in (got, plain))
        assert far <= 2 * allowed + (0.0 if n == "losses" else 2.0 ** -9) * float(want.norm()), (n, far, allowed, float(want.norm()))
