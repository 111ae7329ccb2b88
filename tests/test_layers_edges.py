"""What the binding of the layer operators and of the scan refuses on the host, before anything runs."""

import ctypes
import os
import subprocess

import pytest
import torch
import torch.autograd.forward_ad as fwd

from selective_state_space_29_amd import layers, scan
from test_layers_abi import UNSUPPORTED, gated


def operators():
    """Each differentiable form and its floating-point inputs (on the CPU: a call that is not refused says so)."""
    x, ids = torch.randn(2, 5, 8), torch.randint(0, 9, (2, 5))
    xb, wb = torch.randn(4, 8).bfloat16(), torch.randn(6, 8).bfloat16()
    return [
        (lambda x, r, i, lam, h0: layers.gated_scan(x, r, i, lam, h0=h0), (x, x, x, torch.randn(8), torch.randn(2, 8))),
        (lambda x, w, b, res: layers.layer_norm(x, w, b, residual=res), (x, torch.randn(8), torch.randn(8), x)),
        (lambda w: layers.embedding(ids, w), (torch.randn(9, 8),)),
        (lambda x, g, u: layers.gated_ffn(x, g, u), (xb, wb, wb)),
    ]


@pytest.mark.parametrize("which", range(4))
def test_forward_mode_tangents_are_refused(which):
    f, inputs = operators()[which]
    for k in range(len(inputs)):
        for grad in (False, True):
            with fwd.dual_level():
                given = list(inputs)
                given[k] = fwd.make_dual(inputs[k].clone().requires_grad_(grad), torch.ones_like(inputs[k]))
                with pytest.raises(NotImplementedError, match="forward-mode"):
                    f(*given)
                with torch.no_grad(), pytest.raises(NotImplementedError, match="forward-mode"):
                    f(*given)
    with fwd.dual_level(), pytest.raises(ValueError, match="GPU"):  # a dual level without tangents is no reason
        f(*inputs)


def test_forward_mode_tangents_of_the_scan_are_refused():
    u, A, B = torch.randn(2, 4, 6), -torch.rand(4, 3), torch.randn(2, 3, 6)
    inputs = [u, torch.rand(2, 4, 6), A, B, B.clone(), torch.randn(4), u.clone(), torch.randn(4)]
    for k in range(len(inputs)):
        with fwd.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
            given = list(inputs)
            given[k] = fwd.make_dual(inputs[k], torch.ones_like(inputs[k]))
            scan.selective_scan(*given)


@pytest.mark.parametrize("grad", [False, True])
def test_gated_scan_of_two_dimensions_is_refused_by_its_shape(grad):
    x = torch.randn(5, 8, requires_grad=grad)
    with pytest.raises(ValueError, match="GPU" if not grad else "batch, len, dim"):
        layers.gated_scan(x, x, x, torch.randn(8))


def test_workgroups_take_every_item_once_and_the_xcds_the_same_number(tmp_path):
    """The placement of the recurrence's workgroups, built as host code: XCD k has the workgroups k, k + 8, ..."""
    csrc = os.path.join(os.path.dirname(layers.__file__), "csrc")
    src, lib = tmp_path / "place.cpp", tmp_path / "place.so"
    src.write_text('#include "xcd.hpp"\nextern "C" int64_t place(int64_t id, int64_t n) { return mscan::xcd_item(id, n); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", csrc, "-o", str(lib), str(src)], check=True)
    place = ctypes.CDLL(str(lib)).place
    place.restype, place.argtypes = ctypes.c_int64, [ctypes.c_int64, ctypes.c_int64]
    for n in [*range(1, 70), 192, 240, 252, 256, 257, 288, 1000, 4099]:
        items = [[place(k, n) for k in range(xcd, n, 8)] for xcd in range(8)]
        assert sorted(sum(items, [])) == list(range(n)), n
        assert max(map(len, items)) - min(map(len, items)) <= 1, n
        for own in items:
            assert own == list(range(own[0], own[0] + len(own))) if own else True, n
    # a chain of 64 channels shared by 256 workgroups: 32 of them on every XCD
    assert [place(xcd, 256) // 32 for xcd in range(8)] == list(range(8))


@pytest.mark.parametrize("bwd", [False, True])
def test_gated_limit_counts_groups_of_channels(bwd):
    assert gated(shape=((1 << 23) - 8, 9, 1), bwd=bwd) == UNSUPPORTED  # a narrow row is a whole group
    assert gated(shape=(1 << 18, 9, 1985), bwd=bwd) == UNSUPPORTED     # 32 groups a row
