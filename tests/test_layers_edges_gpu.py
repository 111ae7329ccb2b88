"""The layer operators at their edges: NaN in gates, decays and initial states of packed sequences, and the
accuracy of the recurrence's fp32 results.

A sequence that begins with a reset neither sees what lies before it nor passes a gradient there, so a bad
value is judged against the clean call: where it reaches, NaN; everywhere else the same bits.
"""

import ctypes

import pytest
import torch

from selective_state_space_29_amd import layers
from test_layers_gpu import check_gated, dev, gated_case

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16

# short calls; sequences of one workgroup, in few and in many channels; sequences shared by workgroups
PACKED = [(2, 6, 20), (2, 300, 20), (24, 300, 600), (2, 3000, 70), (1, 5100, 33)]


def packed(B, L, D, dtype, seed=0):
    """Inputs, and resets inside runs, at their ends and at the ends of chunks, up to 3 apart."""
    g = torch.Generator().manual_seed(seed + L + D)
    t = {k: torch.randn(B, L, D, generator=g).to(dtype).to(DEV) for k in ("x", "r", "i", "dy")}
    t["lam"], t["h0"] = torch.randn(D, generator=g).to(DEV), torch.randn(B, D, generator=g).to(DEV)
    at = [k for k in (3, 37, 40, 128, 131, 200, 255, 256, 272, 1000, 1024, 2047, 2048, 2999, 4097) if k < L]
    reset = torch.zeros(B, L, dtype=torch.bool, device=DEV)
    reset[:, at] = True
    return t, reset, at


def run(t, reset, bwd=True):
    kw = dict(h0=t["h0"], reset=reset)
    y, last = layers.gated_scan_fn(t["x"], t["r"], t["i"], t["lam"], return_last_state=True, **kw)
    out = {"y": y, "last": last}
    if bwd:
        ck = torch.empty(layers.gated_checkpoint_shape(*t["x"].shape), device=DEV)
        layers.gated_scan_fn(t["x"], t["r"], t["i"], t["lam"], checkpoints_out=ck, **kw)
        g = layers.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], checkpoints=ck, **kw)
        again = layers.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], **kw)
        for k in g:
            assert torch.equal(g[k].nan_to_num(9e9), again[k].nan_to_num(9e9)) and torch.equal(g[k].isnan(), again[k].isnan()), k
        out |= {"d" + k: v for k, v in g.items()}
    return out


def judge(got, clean, bad):
    for k, v in got.items():
        mask = bad.get(k, torch.zeros_like(v, dtype=torch.bool))
        assert torch.equal(v.isnan(), mask), (k, (v.isnan() != mask).nonzero()[:4].tolist())
        assert torch.equal(v[~mask], clean[k][~mask]), k


def masks(out):
    return {k: torch.zeros_like(v, dtype=torch.bool) for k, v in out.items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D", PACKED)
def test_gated_nan_gate_reaches_its_packed_sequence_alone(B, L, D, dtype):
    t, reset, at = packed(B, L, D, dtype)
    clean = run(t, reset)
    ends = [0, *at, L]
    for k in [k for k in (1, 5, 38, 99, 127, 199, 257, 290, 999, 2046, 2500, 5050) if k < L and k not in at]:
        s = max(e for e in ends if e <= k)          # its sequence is s .. e - 1
        e = min(e for e in ends if e > k)
        first = s not in at                         # the call's first sequence goes on from h0
        b, d = B - 1, (7 * k) % D
        for quiet in (False, True):                 # no gradient from the bad step on: 0 times NaN is NaN too
            u = dict(t, r=t["r"].clone(), dy=t["dy"].clone())
            if quiet:
                u["dy"][b, k:e, d] = 0
                want = run(u, reset)
            else:
                want = clean
            u["r"][b, k, d] = float("nan")
            got = run(u, reset)
            m = masks(got)
            m["y"][b, k:e, d] = True
            m["last"][b, d] = e == L
            m["dx"][b, s:k + 1, d] = m["di"][b, s:k + 1, d] = True
            m["dr"][b, s if first else s + 1:e, d] = True
            m["dh0"][b, d] = first
            m["dlam"][d] = True
            judge(got, want, m)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D", PACKED)
def test_gated_nan_decay_parameter_and_initial_state_with_resets(B, L, D, dtype):
    t, reset, at = packed(B, L, D, dtype, 1)
    clean = run(t, reset)
    on = reset[0]
    d = D // 2
    u = dict(t, lam=t["lam"].clone())
    u["lam"][d] = float("nan")
    got = run(u, reset)
    m = masks(got)
    m["y"][..., d] = ~reset                         # a reset step's state does not depend on its decay
    m["last"][:, d] = not bool(on[-1])
    alone = on & torch.cat([on[1:], torch.ones(1, dtype=torch.bool, device=DEV)])  # sequences of one step
    m["dx"][..., d] = m["di"][..., d] = ~alone      # a reset step's gradient comes through the decay after it
    m["dr"][..., d] = ~reset
    m["dh0"][:, d] = m["dlam"][d] = True
    judge(got, clean, m)

    u = dict(t, h0=t["h0"].clone())
    u["h0"][0, d] = float("nan")
    got = run(u, reset)
    m = masks(got)
    m["y"][0, :at[0], d] = m["dr"][0, :at[0], d] = m["dlam"][d] = True
    judge(got, clean, m)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D", PACKED)
def test_gated_reset_step_does_not_look_at_its_gate(B, L, D, dtype):
    t, reset, at = packed(B, L, D, dtype, 2)
    clean = run(t, reset)
    u = dict(t, r=t["r"].clone())
    u["r"][:, at] = float("nan")
    judge(run(u, reset), clean, {})


@pytest.mark.parametrize("B,L,D", PACKED)
def test_gated_infinite_state_is_forgotten_by_a_reset_alone(B, L, D):
    t, reset, at = packed(B, L, D, F32, 3)
    t["lam"].fill_(8.0)                             # decays of about e^-32 sigmoid(r) a step: a run's vanish in fp32
    clean = run(t, reset, bwd=False)
    t["h0"][0, 3] = float("inf")
    got = run(t, reset, bwd=False)
    assert not got["y"][0, :at[0], 3].isfinite().any()
    got["y"][0, :at[0], 3] = clean["y"][0, :at[0], 3]
    assert torch.equal(got["y"], clean["y"]) and torch.equal(got["last"], clean["last"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [1, 8, 9, 300, 700])
def test_gated_states_are_fp32_whatever_the_activations(L, dtype):
    """A state that is one step's input alone: sqrt(1 - a^2), at small decays, where 1 - a^2 cancels.

    v = -2 log a = 2 c softplus(0) sigmoid(r) between 2^-8 and 2^-3, |r| <= 1. In units of 2^-24: c log2(e)
    softplus 4, exp 3 (its argument's rounding and 1 ulp), 1 + exp 1, its reciprocal 2, the product 1: e errs by
    11 of itself; 1 - a^2 by that and 3 of its own, and its root by half, 7, and 2 for itself. sigmoid(30) rounds
    to 1 within 2^-24, two products: 12 in all.
    """
    D = 2048
    c = (2.0 ** -8 * 32 ** torch.linspace(0, 1, 40, dtype=torch.float64) / (2 * 0.6931 * 0.7)).float()
    r = (2 * torch.rand(40, 1, L, D, generator=torch.Generator().manual_seed(L)) - 1).to(dtype)
    x = torch.zeros(1, L, D, dtype=dtype, device=DEV)
    x[:, -1] = 1
    i, lam = torch.full_like(x, 30.0), torch.zeros(D, device=DEV)
    for k in range(40):
        v = 2 * float(c[k]) * torch.log(torch.tensor(2.0, dtype=torch.float64)) * torch.sigmoid(r[k, 0, -1].double())
        want = torch.sqrt(-torch.expm1(-v))
        _, last = layers.gated_scan_fn(x, r[k].to(DEV), i, lam, c=float(c[k]), return_last_state=True)
        assert float(((last[0].cpu().double() - want) / want).abs().max()) <= 12 * 2.0 ** -24
        if L == 300:                                # the state after step 127, saved for the backward
            u = torch.zeros_like(x)
            u[:, 127] = 1
            ck = torch.empty(layers.gated_checkpoint_shape(1, L, D), device=DEV)
            layers.gated_scan_fn(u, r[k].to(DEV), i, lam, c=float(c[k]), checkpoints_out=ck)
            v = 2 * float(c[k]) * torch.log(torch.tensor(2.0, dtype=torch.float64)) * torch.sigmoid(r[k, 0, 127].double())
            want = torch.sqrt(-torch.expm1(-v))
            assert float(((ck[0, 1].cpu().double() - want) / want).abs().max()) <= 12 * 2.0 ** -24


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim", [1, 40, 768, 2048, 9000, 40001])
def test_norm_statistics_of_a_row_with_a_nan(dim, dtype):
    x = torch.randn(5, dim, device=DEV).to(dtype)
    y0, s0 = layers.layer_norm_fn(x, return_stats=True)
    x[3, dim // 2] = float("nan")
    y, s = layers.layer_norm_fn(x, return_stats=True)
    keep = torch.arange(5, device=DEV) != 3
    assert y[3].isnan().all() and s[3].isnan().all()
    assert torch.equal(y[keep], y0[keep]) and torch.equal(s[keep], s0[keep])


def test_norm_statistics_of_rows_without_columns():
    stale = torch.full((1000, 2), 7.0, device=DEV)
    del stale
    x = torch.zeros(1000, 0, device=DEV)
    y, s = layers.layer_norm_fn(x, return_stats=True)
    assert y.shape == (1000, 0) and s.isnan().all()
    (y, t), s = layers.layer_norm_fn(x, residual=x, return_stats=True)
    assert y.shape == t.shape == (1000, 0) and s.isnan().all()
    g = layers.layer_norm_bwd(x, None, x, s)
    assert g["x"].shape == (1000, 0) and g["weight"].shape == g["bias"].shape == (0,)


# Few chains of 64 channels, each shared by workgroups on one XCD or several; more than 16 chunks, whose states
# pass on by blocks; a last chunk and a last group of channels that are cut short.
SHARED = [(1, 9001, 40), (1, 5001, 70), (2, 2777, 130), (1, 4400, 576), (3, 1500, 200), (2, 700, 70)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("reset", [False, True])
@pytest.mark.parametrize("B,L,D", SHARED)
def test_gated_shared_sequences(B, L, D, reset, dtype):
    """Against the 64-bit reference, by that test file's bars: forward, and the backward with and without states."""
    check_gated(gated_case(21, B, L, D, dtype, reset=reset))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D", SHARED)
def test_gated_shared_sequences_repeat_bit_for_bit(B, L, D, dtype):
    """Calls on other inputs in between leave their own marks in the same workspace."""
    cases = [dev(gated_case(seed, B, L, D, dtype)) for seed in (22, 23)]

    def once(t):
        y, last = layers.gated_scan_fn(t["x"], t["r"], t["i"], t["lam"], h0=t["h0"], return_last_state=True)
        g = layers.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], h0=t["h0"], dlast_state=t["dlast"])
        return [y, last, *g.values()]

    want = [once(t) for t in cases]
    for _ in range(20):
        for t, w in zip(cases, want):
            for a, b in zip(once(t), w):
                assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,D", SHARED)
def test_gated_shared_prompt_updates_its_state_in_place(B, L, D, dtype):
    t = dev(gated_case(24, B, L, D, dtype))
    args = (t["x"], t["r"], t["i"], t["lam"])
    y, last = layers.gated_scan_fn(*args, h0=t["h0"], return_last_state=True)
    for _ in range(10):
        state = t["h0"].clone()
        y2, same = layers.gated_scan_fn(*args, h0=state, return_last_state=True, last_state_out=state)
        assert same is state and torch.equal(state, last) and torch.equal(y2, y)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_gated_shared_sequences_in_a_replayed_graph(dtype):
    t = dev(gated_case(25, 1, 5001, 70, dtype))

    def calls():
        y, last = layers.gated_scan_fn(t["x"], t["r"], t["i"], t["lam"], h0=t["h0"], return_last_state=True)
        return [y, last, *layers.gated_scan_bwd(t["x"], t["r"], t["i"], t["lam"], t["dy"], h0=t["h0"]).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = calls()
    for k in range(4):
        for name in ("x", "dy"):
            t[name].mul_(-1.25 if k % 2 else 0.8)
        want = [v.clone() for v in calls()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b), k


def test_an_error_of_another_call_is_neither_reported_nor_taken():
    """The runtime keeps a thread's last error until somebody asks for it; here that of a device that is not there."""
    hip = ctypes.CDLL("libamdhip64.so")
    x, ids = torch.randn(2, 9, 16, device=DEV), torch.zeros(2, 9, dtype=torch.int64, device=DEV)
    lam, table = torch.zeros(16, device=DEV), torch.randn(5, 16, device=DEV)
    xb, wb = x[0].bfloat16(), torch.randn(8, 16, device=DEV).bfloat16()
    st, dh = layers.layer_norm_fn(x, return_stats=True)[1], torch.ones(9, 8, device=DEV).bfloat16()
    for f in (lambda: layers.gated_scan_fn(x, x, x, lam), lambda: layers.gated_scan_bwd(x, x, x, lam, x),
              lambda: layers.layer_norm_fn(x), lambda: layers.layer_norm_bwd(x, None, x, st),
              lambda: layers.embedding_fn(ids, table), lambda: layers.embedding_bwd(ids, x, 5),
              lambda: layers.gated_ffn_fn(xb, wb, wb), lambda: layers.gated_ffn_bwd(xb, wb, wb, dh)):
        f()
        torch.cuda.synchronize()
        bad = hip.hipSetDevice(1000)
        assert bad != 0
        try:
            f()
        finally:
            left = hip.hipGetLastError()
        assert left == bad
