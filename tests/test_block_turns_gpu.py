"""Block operators at sizes whose workgroups take several turns over their work, every result and gradient against
64-bit references vectorised over steps; each test states how many turns its sizes make.

Bars. Activations' results: fp32 1e-4 (1 + |r|), the bar of the other tests, and 2^-8 |r| for one rounded to bf16. A
parameter's gradient is a sum in fp32 of terms whose magnitudes the reference adds up as well: a lane's own sum, the
lanes', waves' and workgroups' in their order make fewer than 512 additions one after another, each off by half a unit
of at most the magnitudes' sum, and a term has a few roundings of its own: 2^-24 * 512 of that sum.
"""

import pytest
import torch

import block_ref as ref
from selective_state_space_29_amd import block, scan

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
SUM = 2.0 ** -24 * 512


def within(got, want, room):
    err = (got.double() - want).abs()
    room = room + (2.0 ** -8 * want.abs() if got.dtype == BF16 else 0.0)
    assert bool((err <= room).all()), (float((err - room).max()), int((err - room).argmax()))


def close(got, want):
    within(got, want, 1e-4 * (1 + want.abs()))


def conv_reference(x, weight, bias, state, reset, dy, dlast):
    """(y, last state, gradients, the sums of magnitudes behind the parameters' gradients), in 64 bits."""
    x, weight, bias, state, dy, dlast = (t.double() for t in (x, weight, bias, state, dy, dlast))
    (B, L, D), W = x.shape, weight.shape[1]
    line = torch.cat([state, x], 1)
    at = torch.arange(L + W - 1, device=x.device)
    # the first place of the line that belongs to each place's sequence
    begin = torch.zeros(B, L + W - 1, dtype=torch.int64, device=x.device)
    begin[:, W - 1:] = torch.where(reset, at[W - 1:], 0).cummax(1).values
    seen = [(at[k:k + L] >= begin[:, W - 1:])[..., None] for k in range(W)]
    pre = bias + sum(weight[:, k] * line[:, k:k + L] * seen[k] for k in range(W))
    alive = (at[L:] >= begin[:, -1:])[..., None]
    dpre = dy * ref.dsilu(pre)
    dline = torch.zeros_like(line)
    dline[:, L:] = dlast * alive
    dw, room = [], []
    for k in range(W):
        dline[:, k:k + L] += weight[:, k] * dpre * seen[k]
        terms = dpre * line[:, k:k + L] * seen[k]
        dw.append(terms.sum((0, 1)))
        room.append(terms.abs().sum((0, 1)))
    grads = {"x": dline[:, W - 1:], "initial_state": dline[:, :W - 1], "weight": torch.stack(dw, 1), "bias": dpre.sum((0, 1))}
    return ref.silu(pre), line[:, L:] * alive, grads, {"weight": torch.stack(room, 1), "bias": dpre.abs().sum((0, 1))}


def conv_inputs(seed, B, L, D, W, dtype, device):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
    reset = torch.rand(B, L, generator=g, device=device) < 1 / 150
    return (r(B, L, D).to(dtype), r(D, W) * W ** -0.5, r(D), r(B, W - 1, D).to(dtype), reset, r(B, L, D).to(dtype), r(B, W - 1, D).to(dtype))


def test_the_vectorised_reference_is_the_one_step_by_step():
    for W in (2, 4):
        x, w, b, state, reset, dy, dlast = conv_inputs(1, 2, 9, 3, W, F32, "cpu")
        reset[0, 4] = reset[1, 0] = reset[1, 7] = True
        y, last, grads, _ = conv_reference(x, w, b, state, reset, dy, dlast)
        want_y, want_last, want = ref.causal_conv(x, w, b, state, reset, "silu", dy, dlast)
        assert torch.allclose(y, want_y, 1e-12, 1e-12) and torch.equal(last, want_last)
        assert all(torch.allclose(grads[k], want[k], 1e-12, 1e-12) for k in want)


def gradient_turns(B, L, D, W, dtype, steps):
    """How often the busiest workgroup of the gradient goes round: its runs of 32 - (W - 1) steps, 4 at a time, or of 8
    steps, 252 at a time, over the number of workgroups that the workspace has a row of sums for."""
    n = block._load().mamba_conv_bwd_workspace_bytes(block.ConvShape(B, L, D, W), scan.BF16 if dtype is BF16 else scan.F32, int(steps))
    blocks = n // ((W + 1) * D * 4)
    run, each = (8, 252) if steps else (32 - (W - 1), 4)
    return -(-(B * -(-L // run)) // (each * blocks))


@pytest.mark.gpu
@pytest.mark.parametrize("x_as,y_as,B,L,D,W,dtype", [("rows", "rows", 4, 4000, 4096, 4, BF16), ("rows", "steps", 4, 4000, 4096, 4, BF16),
                                                     ("rows", "rows", 5, 3001, 4001, 3, F32), ("rows", "steps", 5, 3001, 4001, 2, F32),
                                                     ("steps", "steps", 5, 1777, 3001, 4, BF16), ("steps", "steps", 9, 1000, 3002, 3, F32)])
def test_conv_of_several_turns(x_as, y_as, B, L, D, W, dtype):
    """The gradient's workgroups take 4 turns and more; the forward's, of rows, at least 2: runs of 32 steps, 4 at a time, by
    at most 8 workgroups a compute unit over the groups of 128 channels."""
    assert gradient_turns(B, L, D, W, dtype, x_as == "steps") >= 4
    if x_as == "rows":
        cus = torch.cuda.get_device_properties(0).multi_processor_count
        assert B * -(-L // 32) > 4 * (8 * cus // -(-D // 128))
    x, w, b, state, reset, dy, dlast = conv_inputs(B + W, B, L, D, W, dtype, DEV)
    y, last, grads, sums = conv_reference(x, w, b, state, reset, dy, dlast)
    lay = lambda t, how: t.transpose(1, 2).contiguous().transpose(1, 2) if how == "steps" else t  # noqa: E731
    x, dy = lay(x, x_as), lay(dy, y_as)
    kw = dict(initial_state=state, reset=reset)
    got, got_last = block.causal_conv_fn(x, w, b, return_last_state=True, scan_layout=y_as == "steps", **kw)
    close(got, y)
    assert torch.equal(got_last.double(), last)
    del y, got
    g = block.causal_conv_bwd(x, w, b, dy, dlast_state=dlast, **kw)
    for k, want in grads.items():
        within(g[k], want, SUM * sums[k]) if k in sums else close(g[k], want)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,dim,groups", [(40000, 96, 1), (3000, 1536, 1), (3000, 1536, 3), (600, 8000, 1), (40000, 96, 3), (300, 10000, 1)])
def test_norms_of_several_turns(rows, dim, groups, dtype):
    """At most 256 workgroups of 16 waves share the rows of a group: 40000 rows of 96 take 3 turns of 64 rows each (bf16) or 5
    of 32, 3000 of 1536 3 of 4, in 3 groups 3 of 16, 600 of 8000 3 of 1; rows of 10000 are summed by 64 stretches of 5."""
    g = torch.Generator().manual_seed(rows + groups)
    x, z, dy, ds = (torch.randn(rows, dim, generator=g).to(dtype) for _ in range(4))
    w = torch.randn(dim, generator=g)
    d = [t.to(DEV) for t in (x, z, dy, ds, w)]
    n = (x.double() * torch.rsqrt(x.double().square().mean(-1, keepdim=True) + 1e-5)).abs()
    if groups == 1:
        y, stats = block.rms_norm_fn(d[0], d[4], return_stats=True)
        close(y.cpu(), ref.rms_norm(x, w))
        want = ref.rms_norm(x, w, dy=dy, dsum=ds)
        b = block.rms_norm_bwd(d[0], d[4], d[2], stats, dresidual=d[3])
        close(b["x"].cpu(), want["t"])
        within(b["weight"].cpu(), want["weight"], SUM * (dy.double().abs() * n).sum(0))
    for first in (True, False):
        kw = dict(groups=groups, gate_first=first)
        y, stats = block.gated_rms_norm_fn(d[0], d[1], d[4], return_stats=True, **kw)
        close(y.cpu(), ref.gated_rms_norm(x, z, w, **kw))
        want = ref.gated_rms_norm(x, z, w, dy=dy, **kw)
        b = block.gated_rms_norm_bwd(d[0], d[1], d[4], d[2], stats, **kw)
        close(b["x"].cpu(), want["x"])
        close(b["z"].cpu(), want["z"])
        # y before the weight, times dy: what the weight's gradient adds up
        within(b["weight"].cpu(), want["weight"], SUM * (dy.double() * ref.gated_rms_norm(x, z, **kw)).abs().sum(0))
