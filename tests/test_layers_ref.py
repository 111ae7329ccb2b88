"""The references of the layer operators pinned on the CPU: gradients against differences of the
references themselves, and closed forms."""

import pytest
import torch

import layers_ref as ref


def _loss(f, ws):
    out = f()
    return sum((o * w).sum() for o, w in zip(out, ws))


def _differences(f, tensors, grads, ws, step=1e-5):
    """Central differences of the loss in a few single elements of each tensor. The formula's error is
    of fp64 rounding, the differences' about step^2 and 1e-16 / step: 1e-6 relative covers both."""
    g = torch.Generator().manual_seed(5)
    for t, d in zip(tensors, grads):
        for k in torch.randint(0, t.numel(), (6,), generator=g).tolist():
            flat = t.view(-1)
            keep = flat[k].item()
            flat[k] = keep + step
            up = _loss(f, ws)
            flat[k] = keep - step
            down = _loss(f, ws)
            flat[k] = keep
            want = (up - down) / (2 * step)
            assert abs(d.reshape(-1)[k] - want) <= 1e-6 * (1 + abs(want)), (k, d.reshape(-1)[k], want)


@pytest.mark.parametrize("reset", [False, True])
def test_gated_gradient_is_the_differences(reset):
    g = torch.Generator().manual_seed(1)
    B, L, D = 2, 9, 3
    x, r, i, dy = (torch.randn(B, L, D, generator=g, dtype=torch.float64) for _ in range(4))
    lam, h0, dl = torch.randn(D, generator=g, dtype=torch.float64), *(torch.randn(B, D, generator=g, dtype=torch.float64) for _ in range(2))
    rs = torch.rand(B, L, generator=g) < 0.3 if reset else None
    out = ref.gated_scan_bwd(x, r, i, lam, dy, 2.0, h0, rs, dl)
    _differences(lambda: ref.gated_scan(x, r, i, lam, 2.0, h0, rs), (x, r, i, lam, h0),
                 [out[k] for k in ("x", "r", "i", "lam", "h0")], (dy, dl))


def test_gated_closed_forms():
    # gates constant: a geometric series; a reset everywhere: y = sigmoid(i) x
    x, r = torch.full((1, 50, 1), 2.0), torch.zeros(1, 50, 1)
    lam = ref.lam_for(torch.tensor([0.81]))
    y, last = ref.gated_scan(x, r, r, lam)
    a = 0.9  # the gate half open: sqrt(0.81)
    m = (1 - a * a) ** 0.5
    want = [m * (1 - a ** (t + 1)) / (1 - a) for t in range(50)]
    assert torch.allclose(y[0, :, 0], torch.tensor(want, dtype=torch.float64), rtol=1e-6)
    assert last[0, 0] == y[0, -1, 0]
    y, _ = ref.gated_scan(x, r, r, lam, reset=torch.ones(1, 50, dtype=torch.bool))
    assert torch.equal(y, torch.ones_like(y))


def test_norm_gradient_is_the_differences():
    g = torch.Generator().manual_seed(2)
    t, dy, dr = (torch.randn(4, 7, generator=g, dtype=torch.float64) for _ in range(3))
    w, b = (torch.randn(7, generator=g, dtype=torch.float64) for _ in range(2))
    out = ref.layer_norm_bwd(t, w, dy, dresidual=dr)
    _differences(lambda: (ref.layer_norm(t, w, b), t.clone()), (t, w, b), [out[k] for k in ("x", "weight", "bias")], (dy, dr))


def test_embedding_gradient_is_the_differences():
    g = torch.Generator().manual_seed(3)
    ids = torch.tensor([[1, 1, 4], [-1, 0, 9]])
    w, dy = torch.randn(5, 3, generator=g, dtype=torch.float64), torch.randn(2, 3, 3, generator=g, dtype=torch.float64)
    _differences(lambda: (ref.embedding(ids, w, 1.5),), (w,), [ref.embedding_bwd(ids, dy, 5, 1.5)], (dy,))


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
def test_ffn_gradient_is_the_differences(kind):
    g = torch.Generator().manual_seed(4)
    x, wg, wu, dh = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((4, 6), (5, 6), (5, 6), (4, 5)))
    out = ref.gated_ffn_bwd(x, wg, wu, dh, kind)
    _differences(lambda: (ref.gated_ffn(x, wg, wu, kind),), (x, wg, wu), [out[k] for k in ("x", "w_gate", "w_up")], (dh,))
