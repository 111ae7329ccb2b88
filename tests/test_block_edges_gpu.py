"""The block operators at the far ends of what they accept: launches of 2^32 threads and more, sizes whose workgroups
take several turns, rows that lie far apart, the last digits of losses and gradients, outputs that autograd has saved.

Bars stand beside the tests that need one; elsewhere results are the bits of a smaller call by the same kernels.
"""

import pytest
import torch

from selective_state_space_29_amd import block

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16


def gen(seed):
    return torch.Generator().manual_seed(seed)


def stale(*shape):
    """Memory that holds 99 where a result is going to lie: what an unwritten row would show."""
    t = torch.full(shape, 99.0, device=DEV)
    del t


def over(t, n):
    """n rows: t's, over and over (indexing so many rows with a tensor loses some in torch itself)."""
    return t.repeat(-(-n // t.shape[0]), *[1] * (t.dim() - 1))[:n]


def test_cross_entropy_more_rows_than_a_grid_counts_threads():
    rows, few = (1 << 26) + 1000, 251  # the join of a row's tiles takes 64 threads a row
    g = gen(1)
    x, w = torch.randn(few, 8, generator=g).to(BF16).to(DEV), torch.randn(5, 8, generator=g).to(BF16).to(DEV)
    t = torch.randint(-1, 6, (few,), generator=g, dtype=torch.int32).to(DEV)
    small = block.linear_cross_entropy_fn(x, w, t, return_lse=True)
    X, T = over(x, rows), over(t, rows)
    stale(2, rows)
    loss, lse = block.linear_cross_entropy_fn(X, w, T, return_lse=True)
    assert torch.equal(loss, over(small[0], rows)) and torch.equal(lse, over(small[1], rows))
    del loss
    want = block.linear_cross_entropy_bwd(x, w, t, small[1], torch.ones(few, device=DEV), want_dweight=False)["x"]
    got = block.linear_cross_entropy_bwd(X, w, T, lse, torch.ones(1, device=DEV).expand(rows), want_dweight=False)["x"]
    assert torch.equal(got, over(want, rows))


def test_step_of_more_sums_than_a_grid_counts_threads():
    batch, few, rank = 1 << 23, 97, 512  # a thread for each of the 514 sums of a stream
    g = gen(2)
    r = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    t = dict(x=r(few, 1), conv_state=r(few, 1, 1), ssm_state=r(few, 1, 1))
    weights = dict(conv_w=r(1, 2), conv_b=r(1), w_x=r(rank + 2, 1), w_dt=r(1, rank) * rank ** -0.5, dt_bias=r(1), A=-torch.ones(1, 1, device=DEV))
    many = {k: over(v, batch) for k, v in t.items()}
    y = block.block_step(**t, **weights)
    stale(batch, rank)
    got = block.block_step(**many, **weights)
    assert torch.equal(got, over(y, batch)) and torch.equal(many["ssm_state"], over(t["ssm_state"], batch))
