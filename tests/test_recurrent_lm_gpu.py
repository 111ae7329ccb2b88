"""The example language model: its gradients against the same model on plain operators, and decoding
token by token against the whole sequence at once.

Bars. Every operator rounds its result to bf16, 2^-8 of it at most, and a value passes through about 11
of them a block, so two ways of rounding agree to about 2^-8 * 11 * depth of a tensor's norm, in a
gradient twice that (the way forward and back).
"""

import importlib.util
import os
import sys

import pytest
import torch
import torch.nn.functional as F

from selective_state_space_29_amd import layers

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_lm.py")
DEPTH = 2


def example():
    spec = importlib.util.spec_from_file_location("recurrent_lm", PATH)
    mod = importlib.util.module_from_spec(spec)
    sys.modules["recurrent_lm"] = mod
    spec.loader.exec_module(mod)
    return mod


def small_model(ex):
    torch.manual_seed(1)
    return ex.RecurrentLM(50, 72, DEPTH, 100).cuda()


class Plain:
    """The four operators from elementary torch operations, rounded to bf16 where theirs are."""

    @staticmethod
    def gated_scan(x, r, i, lam, reset=None, c=8.0):
        log_a = -c * F.softplus(lam) * torch.sigmoid(r.float())
        a = torch.exp(log_a) * (1 if reset is None else (~reset)[..., None])
        b = torch.sqrt(1 - a * a) * torch.sigmoid(i.float()) * x.float()
        h, out = torch.zeros_like(b[:, 0]), []
        for t in range(x.shape[1]):
            h = a[:, t] * h + b[:, t]
            out.append(h)
        return torch.stack(out, 1).to(x.dtype)

    @staticmethod
    def layer_norm(x, weight, bias, residual=None):
        t = x if residual is None else x + residual
        y = F.layer_norm(t.float(), t.shape[-1:], weight, bias).to(x.dtype)
        return y if residual is None else (y, t)

    @staticmethod
    def embedding(ids, w, scale):
        return (w.float()[ids] * scale).to(w.dtype)

    @staticmethod
    def gated_ffn(x, wg, wu):
        x, wg, wu = x.float(), wg.float(), wu.float()
        return (F.silu(x @ wg.t()) * (x @ wu.t())).bfloat16()


def near(got, want, room):
    err = float((got.double() - want.double()).norm())
    assert err <= room * float(want.double().norm()), (err, float(want.double().norm()))


def test_training_step_matches_plain_operators():
    ex = example()
    model = small_model(ex)
    ids, reset = ex.documents(3, 150, 50, "cuda", torch.Generator().manual_seed(2))
    loss = model.loss(ids, reset)
    loss.backward()
    got = {n: p.grad.clone() for n, p in model.named_parameters()}
    model.zero_grad()
    ex.layers = Plain
    want = model.loss(ids, reset)
    want.backward()
    near(loss.detach(), want.detach(), 2.0 ** -8 * 11 * DEPTH)
    for n, p in model.named_parameters():
        assert got[n].dtype == p.dtype
        near(got[n], p.grad, 2 * 2.0 ** -8 * 11 * DEPTH)


def test_decoding_continues_the_sequence():
    ex = example()
    model = small_model(ex)
    ids, _ = ex.documents(4, 90, 50, "cuda", torch.Generator().manual_seed(3))
    with torch.no_grad():
        whole = model(ids)
        states = model.new_states(4)
        parts = [model(ids[:, :37], states=states)] + [model(ids[:, k:k + 1], states=states) for k in range(37, 90)]
    near(torch.cat(parts, 1), whole, 2.0 ** -8 * 11 * DEPTH)


def test_captured_decoding_step_repeats_the_eager_one():
    ex = example()
    model = small_model(ex)
    ids, _ = ex.documents(5, 20, 50, "cuda", torch.Generator().manual_seed(4))
    eager, graph = ex.Decoder(model, 5), ex.Decoder(model, 5)
    graph.capture()
    for d in (eager, graph):
        d.prompt(ids)
    for k in range(12):  # replays between eager steps and waits
        a, b = eager.generate(1), graph.generate(1)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and torch.equal(eager.logits, graph.logits), k
        for s, t in zip(eager.states, graph.states):
            assert torch.equal(s, t), k


def test_learns_to_count():
    ex = example()
    torch.manual_seed(0)
    model = ex.RecurrentLM(32, 96, 2, 200).cuda()
    optimizer = torch.optim.AdamW(model.parameters(), lr=2e-3, weight_decay=0.0)
    g = torch.Generator().manual_seed(5)
    losses = []
    for _ in range(60):
        loss = model.loss(*ex.documents(16, 256, 32, "cuda", g))
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    assert losses[-1] < 0.5 * losses[0], losses[::10]


def test_second_derivatives_are_refused():
    x = torch.randn(2, 8, device="cuda", requires_grad=True)
    (g,) = torch.autograd.grad(layers.layer_norm(x).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
