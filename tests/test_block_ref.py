"""The block operators' references themselves: gradients against differences, and the measured plain forms'
definitions against them (CPU)."""

import pytest
import torch

import block_ref as ref


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, dtype=torch.float64)


def against_differences(f, inputs, grads, names):
    """Each gradient along a random direction against a central difference of f."""
    g = gen(99)
    for k, name in enumerate(names):
        v = randn(g, *inputs[k].shape)
        at = lambda e: f(*[t + e * v if i == k else t for i, t in enumerate(inputs)])  # noqa: E731
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        want = (grads[name] * v).sum()
        assert abs(float(diff - want)) <= 1e-7 * (1 + abs(float(want))), name


@pytest.mark.parametrize("activation", ["silu", None])
@pytest.mark.parametrize("width", [1, 2, 3, 4])
@pytest.mark.parametrize("length", [1, 2, 9])
def test_causal_conv_gradients(width, length, activation):
    g = gen(width * 10 + length)
    B, D = 2, 3
    x, w, b, s = randn(g, B, length, D), randn(g, D, width), randn(g, D), randn(g, B, width - 1, D)
    reset = torch.rand(B, length, generator=g) < 0.3
    dy, dl = randn(g, B, length, D), randn(g, B, width - 1, D)

    def loss(x, w, b, s):
        y, last = ref.causal_conv(x, w, b, s, reset, activation)
        return (y * dy).sum() + (last * dl).sum()

    grads = ref.causal_conv(x, w, b, s, reset, activation, dy, dl)[2]
    against_differences(loss, [x, w, b, s], grads, ["x", "weight", "bias", "initial_state"])


def test_causal_conv_is_a_padded_convolution():
    g = gen(3)
    x, w, b = randn(g, 2, 11, 5), randn(g, 5, 4), randn(g, 5)
    y, last = ref.causal_conv(x, w, b, activation=None)
    want = torch.nn.functional.conv1d(torch.nn.functional.pad(x.transpose(1, 2), (3, 0)), w[:, None], b, groups=5).transpose(1, 2)
    assert torch.allclose(y, want, rtol=0, atol=1e-12)
    assert torch.equal(last, x[:, -3:])


def test_causal_conv_pieces_are_the_whole():
    g = gen(4)
    x, w = randn(g, 2, 12, 3), randn(g, 3, 4)
    reset = torch.zeros(2, 12, dtype=torch.bool)
    reset[0, 5] = reset[1, 6] = True
    y, last = ref.causal_conv(x, w, reset=reset)
    state, parts = None, []
    for s in (slice(0, 1), slice(1, 6), slice(6, 8), slice(8, 12)):
        part, state = ref.causal_conv(x[:, s], w, state=state, reset=reset[:, s])
        parts.append(part)
    # (the CPU's exponentials of a tensor's last few values may take another path: a few units in the last place)
    assert torch.allclose(torch.cat(parts, 1), y, rtol=0, atol=1e-14) and torch.equal(state, last)


def test_rms_norm_gradients():
    g = gen(5)
    t, w, dy, ds = randn(g, 4, 9), randn(g, 9), randn(g, 4, 9), randn(g, 4, 9)
    grads = ref.rms_norm(t, w, dy=dy, dsum=ds)
    against_differences(lambda t, w: (ref.rms_norm(t, w) * dy).sum() + (t * ds).sum(), [t, w], grads, ["t", "weight"])


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("groups", [1, 3])
def test_gated_rms_norm_gradients(groups, gate_first):
    g = gen(6)
    x, z, w, dy = randn(g, 4, 12), randn(g, 4, 12), randn(g, 12), randn(g, 4, 12)
    kw = dict(groups=groups, gate_first=gate_first)
    grads = ref.gated_rms_norm(x, z, w, dy=dy, **kw)
    against_differences(lambda x, z, w: (ref.gated_rms_norm(x, z, w, **kw) * dy).sum(), [x, z, w], grads, ["x", "z", "weight"])


def test_linear_cross_entropy_gradients():
    g = gen(7)
    x, w = randn(g, 6, 5), randn(g, 11, 5)
    target = torch.tensor([0, 10, -100, 3, 11, 3])
    dloss, dlse = randn(g, 6), randn(g, 6)

    def f(x, w):
        loss, lse = ref.linear_cross_entropy(x, w, target, 0.7)
        return (loss * dloss).sum() + (lse * dlse).sum()

    against_differences(f, [x, w], ref.linear_cross_entropy(x, w, target, 0.7, dloss, dlse)[2], ["x", "weight"])
    loss, _ = ref.linear_cross_entropy(x, w, target)
    want = torch.nn.functional.cross_entropy(x @ w.t(), target.masked_fill(target == 11, -100), reduction="none", ignore_index=-100)
    assert torch.allclose(loss, want, rtol=0, atol=1e-12)
