"""Host-only checks of the block operators' workspace sizes: what a call does not need is not asked for. No call is
made; pointers are made-up addresses that are never followed."""

import pytest

from selective_state_space_29_amd import block, scan

BASE = 1 << 40


FACTORS = 256 + 256 * 16  # the rows' common factor and what it is found from


def up(n, a=256):
    return -(-n // a) * a


def xent_bwd(rows, dim, vocab, dx=True, dweight=True):
    p = block.XentBwdPtrs(x=BASE, weight=BASE * 2, target=BASE * 3, lse=BASE * 4, dloss=BASE * 5, dx=BASE * 6 if dx else None,
                          dweight=BASE * 7 if dweight else None, x_stride=dim, weight_stride=dim, dloss_stride=1)
    return block._load().mamba_xent_bwd_workspace_bytes(p, block.XentShape(rows, dim, vocab))


@pytest.mark.parametrize("rows,dim,vocab", [(16384, 768, 50000), (16384, 64, 9000), (300, 64, 1000)])
def test_cross_entropy_gradients_that_are_not_asked_for_take_no_room(rows, dim, vocab):
    both, dx, dw, none = (xent_bwd(rows, dim, vocab, a, b) for a, b in ((1, 1), (1, 0), (0, 1), (0, 0)))
    # of each row its factors and its part of x; at most 256 MB of the logits' gradients and a piece's rounding
    base = up(rows * 16) + FACTORS + up(rows * dim * 2)
    assert base < none <= base + (1 << 28) + rows * 512
    assert both - none == (dx - none) + (dw - none)
    if rows == 16384:  # several pieces: dx's sums in fp32; the parts of dweight's sums
        assert dx - none >= rows * dim * 4 and dw - none > 0


@pytest.mark.parametrize("rows,vocab,pieces", [(16384, 32768, 4), (8192, 32768, 2), (16384, 32769, 5), (16384, 8192, 1), (1 << 18, 100000, 98)])
def test_cross_entropy_pieces_are_as_many_as_their_bytes_ask_for(rows, vocab, pieces):
    """256 MB of the logits' gradients a piece, of 1024 columns at least and a multiple of 256."""
    dim = 64
    width = max(1024, up(-(-vocab // pieces)))
    assert xent_bwd(rows, dim, vocab, False, False) == up(rows * 16) + FACTORS + up(rows * dim * 2) + up(rows * width * 2)


@pytest.mark.parametrize("rows,dim", [(1, 1 << 20), (3, 1001), (100, 64), (256, 768), (16384, 1536)])
def test_norm_gradients_ask_for_no_more_partial_sums_than_rows(rows, dim):
    lib = block._load()
    most = up(min(rows, 256) * dim * 4)
    assert lib.mamba_rms_norm_bwd_workspace_bytes(block.RmsShape(rows, dim)) == most
    assert lib.mamba_gated_rms_norm_bwd_workspace_bytes(block.GatedRmsShape(rows, dim, 1)) == most


@pytest.mark.parametrize("steps", [0, 1])
def test_conv_takes_as_many_runs_as_the_header_says(steps):
    size = lambda *s: block._load().mamba_conv_bwd_workspace_bytes(block.ConvShape(*s), scan.BF16, steps)  # noqa: E731
    for batch, length in ((1 << 30, 8), ((1 << 31) - 1, 1), ((1 << 31) - 1, 0), ((1 << 30) - 1, 9), (1, (1 << 30) - 1)):
        assert size(batch, length, 1, 4) > 0, (batch, length)
    for batch, length in ((1 << 30, 9), (1 << 31, 0), (1, 1 << 30), (1 << 27, 128)):
        assert size(batch, length, 1, 4) < 0, (batch, length)


def test_what_is_not_supported_is_not_blamed_on_a_forced_kernel_alone():
    """The entry points without kernels to force refuse by the same code: fp32 in the cross entropy, sizes past a limit."""
    p = block.XentPtrs(x=BASE, weight=BASE * 2, target=BASE * 3, loss=BASE * 4, x_stride=8, weight_stride=8)
    code = block._load().mamba_xent_fwd(p, block.XentShape(4, 8, 9), 1, 1.0, scan.F32, None)
    assert code == -8 and "entry point" in scan.strerror(code) and "type" in scan.strerror(code)
