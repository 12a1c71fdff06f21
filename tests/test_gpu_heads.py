"""The head scan (linear attention with one decay per head) against the recurrence in 64 bits: packed
prefill, single tokens, gradients.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import heads_ref as ref
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

KEYS = ("proj", "cu", "A_log", "D", "dt_bias", "state", "dy", "dstate")


def to_gpu(c):
    g = dict(c)
    for k in KEYS:
        g[k] = c[k].cuda() if c[k] is not None else None
    return ref.split(g, c["dt"] is not None)


def tokens(g):
    return [g[k] for k in ("x", "dt", "B", "C", "A_log", "D", "dt_bias")]


# lens, H, P, G, N, io, and which optional arguments are absent
CASES = [
    ([1], 1, 1, 1, 1, "f32", ""),
    ([1], 4, 64, 1, 128, "bf16", ""),
    ([0, 3, 0], 3, 5, 3, 7, "f32", "D"),
    ([64], 2, 64, 1, 128, "bf16", ""),
    ([65, 63, 1, 128, 0, 200], 4, 64, 2, 128, "bf16", ""),
    ([130, 17], 6, 40, 3, 24, "bf16", "dt"),
    ([100, 31], 2, 80, 1, 100, "bf16", "state"),
    ([77, 200], 3, 128, 1, 64, "bf16", "D"),
    ([77, 90], 5, 20, 5, 50, "bf16", ""),
    ([129], 2, 256, 1, 256, "bf16", ""),
    ([70, 60], 2, 33, 1, 200, "f32", "dt state"),
    ([129, 64, 5], 4, 64, 2, 128, "f32", ""),
    ([50, 150], 8, 16, 2, 16, "bf16", ""),
]
IDS = [f"{'-'.join(map(str, c[0]))}_H{c[1]}P{c[2]}G{c[3]}N{c[4]}_{c[5]}_{c[6].replace(' ', '')}" for c in CASES]


def make(case, seed=1):
    lens, H, P, G, N, io, no = case
    return ref.heads_inputs(seed, lens, H, P, G, N, io, "dt" not in no, "D" not in no, "state" not in no)


def run_prefill(c, **kw):
    g = to_gpu(c)
    y, s = mm.heads_prefill(*tokens(g), g["cu"], g["state"], **kw)
    torch.cuda.synchronize()
    return y, s


def check_prefill(c, y, s):
    yr, sr, ya, sa = ref.forward(c)
    T = sum(c["lens"])
    a, b = ref.check(y, yr, ya, T, "y"), ref.check(s, sr, sa, T, "state")
    log(f"  y {a:.2g}, state {b:.2g} of the bound")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_prefill(case):
    c = make(case)
    check_prefill(c, *run_prefill(c))


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_prefill_long_sequences_in_segments(io):
    c = ref.heads_inputs(2, [1900, 3, 1500, 0, 700], 2, 24, 1, 32, io)
    check_prefill(c, *run_prefill(c))


def test_prefill_wide_heads_in_segments():
    c = ref.heads_inputs(3, [2100, 0, 900], 2, 64, 1, 128, "bf16")
    check_prefill(c, *run_prefill(c))


@pytest.mark.parametrize("shape", [(4, 64, 1, 128), (3, 20, 3, 50)])
def test_prefill_in_place_and_in_two_calls(shape):
    """The state carried from one call to the next, updated in place, and the same sequences in one call."""
    H, P, G, N = shape
    lens = [700, 1, 90]
    c = ref.heads_inputs(4, lens, H, P, G, N, "bf16")
    g = to_gpu(c)
    y1, s1 = mm.heads_prefill(*tokens(g), g["cu"], g["state"])
    cut = [300, 0, 64]
    parts = []
    state = g["state"].clone()
    for k in range(2):
        rows = []
        at = 0
        for n, m in zip(lens, cut):
            rows += list(range(at, at + m)) if k == 0 else list(range(at + m, at + n))
            at += n
        part = dict(c, proj=c["proj"][rows], lens=cut if k == 0 else [n - m for n, m in zip(lens, cut)])
        part["cu"] = torch.tensor([sum(part["lens"][:i]) for i in range(4)], dtype=torch.int32)
        p = to_gpu(part)
        y, out = mm.heads_prefill(*tokens(p), p["cu"], state, state_out=state)
        assert out is state
        parts.append((rows, y))
    torch.cuda.synchronize()
    y2 = torch.empty_like(y1)
    for rows, y in parts:
        y2[torch.tensor(rows, device="cuda")] = y
    yr, sr, ya, sa = ref.forward(c)
    ref.check(y2, yr, ya, 800, "y in two calls")
    ref.check(state, sr, sa, 800, "state in place")
    ref.check(s1, sr, sa, 800, "state in one call")


@pytest.mark.parametrize("shape", [(2, 64, 1, 128, "bf16"), (2, 16, 1, 16, "f32")])
def test_large_and_small_steps(shape):
    """delta from 0 to 40 in one sequence: decays that vanish, tokens that barely count, and small steps after
    large ones, whose decays must not be lost in the sum."""
    H, P, G, N, io = shape
    c = ref.heads_inputs(5, [200], H, P, G, N, io)
    g = torch.Generator().manual_seed(9)
    pick = torch.randint(0, 4, c["dt"].shape, generator=g)
    c["dt"].copy_(torch.tensor([-40.0, -5.0, 0.0, 44.0])[pick].to(c["dt"].dtype))
    check_prefill(c, *run_prefill(c))


@pytest.mark.parametrize("shape", [(2, 64, 1, 128, "bf16"), (3, 20, 1, 24, "bf16"), (2, 16, 1, 16, "f32")])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_stay_in_their_sequence_and_after_their_token(shape, value):
    H, P, G, N, io = shape
    c = ref.heads_inputs(6, [90, 100, 40], H, P, G, N, io)
    clean_y, clean_s = run_prefill(c)
    at = 90 + 37
    for key in ("x", "B"):
        d = dict(c, proj=c["proj"].clone())
        ref.split(d)
        d[key][at] = value
        y, s = run_prefill(d)
        assert torch.equal(y[:90], clean_y[:90]) and torch.equal(y[190:], clean_y[190:]), f"{key}: other sequences"
        assert torch.isfinite(y[90:at]).all(), f"{key}: earlier tokens"
        assert (y[90:at].float() - clean_y[90:at].float()).abs().max() <= 0.05 * clean_y.float().abs().max()
        assert torch.equal(s[0], clean_s[0]) and torch.equal(s[2], clean_s[2])
        assert not torch.isfinite(y[at]).all() and not torch.isfinite(s[1]).all()


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_decode(case):
    _, H, P, G, N, io, no = case
    c = ref.heads_inputs(7, [1] * 5, H, P, G, N, io, "dt" not in no, "D" not in no, "state" not in no)
    g = to_gpu(c)
    y, s = mm.heads_decode(*tokens(g), g["state"])
    yr, sr, ya, sa = ref.forward(c)
    # no operand is rounded in the single-token form: the float32 bound and the output's rounding
    tol = ref.F32_EPS * 20 * ya + (2.0 ** -8 * yr.abs() if io == "bf16" else 0)
    assert ((y.cpu().double() - yr).abs() <= tol + 1e-30).all()
    ref.check(s, sr, sa, 1, "state")
    if g["state"] is not None:
        state = g["state"].clone()
        y2, _ = mm.heads_decode(*tokens(g), state, state_out=state)
        assert torch.equal(state, s) and torch.equal(y2, y)


def test_decode_continues_a_prefill():
    c = ref.heads_inputs(8, [40, 1, 64], 4, 64, 2, 128, "bf16")
    lens = [39, 0, 63]
    ends = [39, 40, 104]
    rows = [t for t in range(105) if t not in ends]
    part = dict(c, proj=c["proj"][rows], lens=lens, cu=torch.tensor([0, 39, 39, 102], dtype=torch.int32))
    p, last = to_gpu(part), to_gpu(dict(c, proj=c["proj"][ends]))
    _, s = mm.heads_prefill(*tokens(p), p["cu"], p["state"])
    y, s = mm.heads_decode(*tokens(last), s, state_out=s)
    yr, sr, ya, sa = ref.forward(c)
    ref.check(y, yr[ends], ya[ends], 64, "y")
    ref.check(s, sr, sa, 64, "state")


def test_streams_and_reproducibility():
    """On another stream than the current one, and twice with the same bits."""
    c = ref.heads_inputs(9, [300, 200], 4, 64, 1, 128, "bf16")
    y1, s1 = run_prefill(c)
    side = torch.cuda.Stream()
    g = to_gpu(c)
    torch.cuda.synchronize()
    y2, s2 = mm.heads_prefill(*tokens(g), g["cu"], g["state"], stream=side)
    side.synchronize()
    assert torch.equal(y1, y2) and torch.equal(s1, s2)


GRADS = ("dx", "ddt", "dB", "dC", "dA_log", "dD", "ddt_bias", "dstate_in")


def run_backward(c, **kw):
    g = to_gpu(c)
    out = mm.heads_backward(*tokens(g), g["cu"], g["state"], g["dy"], g["dstate"], **kw)
    torch.cuda.synchronize()
    return out


def check_backward(c, got, dstate=True):
    T = sum(c["lens"])
    want = ref.backward(c, dstate)
    said = []
    for k in GRADS:
        if k not in want:
            assert got[k] is None
            continue
        said.append(f"{k} {ref.check(got[k], *want[k], T, k):.2g}")
    log("  of the bound: " + ", ".join(said))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(case):
    c = make(case, seed=11)
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("shape", [(2, 64, 1, 128, "bf16"), (2, 24, 1, 32, "f32")])
def test_backward_long_sequences_in_segments(shape):
    H, P, G, N, io = shape
    c = ref.heads_inputs(12, [1700, 0, 900, 1], H, P, G, N, io)
    check_backward(c, run_backward(c))


def test_backward_without_a_final_state_gradient_into_column_ranges():
    c = ref.heads_inputs(13, [90, 45], 4, 64, 2, 128, "bf16")
    g = to_gpu(c)
    dproj = torch.zeros_like(g["proj"])
    o = ref.split(dict(c, proj=dproj))
    got = mm.heads_backward(*tokens(g), g["cu"], g["state"], g["dy"], None, dx=o["x"], ddt=o["dt"], dB=o["B"], dC=o["C"])
    check_backward(c, got, dstate=False)
    assert (dproj[:, :256] == 0).all(), "columns that are no gradient were written"


def test_backward_is_reproducible():
    c = ref.heads_inputs(14, [300, 200], 4, 64, 1, 128, "bf16")
    a, b = run_backward(c), run_backward(c)
    for k in GRADS:
        assert torch.equal(a[k], b[k]), k


def test_backward_against_differences():
    """The gradients along a direction against central differences of the 64-bit forward (step 1e-4: its
    truncation, 1e-8 relative to third derivatives of order one, is far below the float32 bound)."""
    c = ref.heads_inputs(15, [33, 70], 3, 12, 3, 10, "f32")
    got = run_backward(c)
    names = dict(x="dx", dt="ddt", B="dB", C="dC", A_log="dA_log", D="dD", dt_bias="ddt_bias", state="dstate_in")
    want = ref.backward(c)
    for k, gk in names.items():
        v = torch.randn(c[k].shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
        loss = []
        for e in (1e-4, -1e-4):
            d = dict(c)
            d[k] = c[k].double() + e * v
            y, s, _, _ = ref.forward(d)
            loss.append(float((y * c["dy"].double()).sum() + (s * c["dstate"].double()).sum()))
        diff = (loss[0] - loss[1]) / 2e-4
        mine = float((got[gk].cpu().double() * v).sum())
        tol = float((ref.bound(*want[gk], torch.float32, 103) * v.abs()).sum()) + 1e-5 * abs(diff)
        assert abs(mine - diff) <= tol, f"{k}: {mine} against {diff}"
