"""The gated recurrence against its definition in 64 bits.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

# lens, d, io: empty and one-token sequences, sequences that start and end at, before and behind a block's border, odd
# channels, many blocks
CASES = [([1], 1, "f32"), ([1, 0, 2, 3, 1], 5, "bf16"), ([255, 1, 257, 0, 30], 64, "bf16"), ([256, 256, 512], 33, "f32"),
         ([300, 5, 0, 1, 77], 130, "f32"), ([1] * 300, 40, "bf16"), ([1030], 250, "bf16"), ([0, 0, 5, 0], 12, "f32"),
         ([10, 700, 3], 97, "bf16"), ([5000, 3, 900], 24, "f32"), ([9300], 32, "bf16"), ([0, 0], 8, "f32")]
# lam, g, z, gate
FORMS = [(True, True, True, "gelu"), (True, False, False, "silu"), (False, False, True, "silu"), (False, True, False, "gelu"),
         (True, True, False, "silu")]


def gpu(t):
    return t.cuda() if t is not None else None


def inputs(c):
    return [gpu(c[k]) for k in ("x", "r", "g", "z", "lam")]


def strided(c):
    """x, r, g, z as column ranges of one tensor on the GPU."""
    d = c["x"].shape[1]
    p = torch.zeros(c["x"].shape[0], 4 * d + 5, dtype=c["x"].dtype, device="cuda")
    out = []
    for i, k in enumerate(("x", "r", "g", "z")):
        if c[k] is not None:
            p[:, i * d:(i + 1) * d] = c[k].cuda()
        out.append(p[:, i * d:(i + 1) * d] if c[k] is not None else None)
    return out + [gpu(c["lam"])]


@pytest.mark.parametrize("lam,g,z,gate", FORMS)
@pytest.mark.parametrize("lens,d,io", CASES)
def test_prefill(lens, d, io, lam, g, z, gate):
    c = ref.gated_inputs(1, lens, d, io, lam, g, z, state=not (z and not lam))
    T = sum(lens)
    y, last, ckpt = mm.gated_prefill_train(*strided(c), c["cu"].cuda(), gpu(c["state"]), gate=gate)
    want, wl, mag, lmag, before = ref.gated(c, gate)
    ref.check(y, want, mag, T, "y")
    ref.check(last, wl, lmag, T, "state")
    ref.check(ckpt, *(t[::mm.layer.GATED_BLOCK] for t in before), T, "checkpoints")
    y2, l2 = mm.gated_prefill(*inputs(c), c["cu"].cuda(), gpu(c["state"]), gate=gate)
    assert torch.equal(y2, y) and torch.equal(l2, last), "rows of another stride, no checkpoints"
    if c["state"] is not None:
        s = c["state"].cuda()
        y3, l3 = mm.gated_prefill(*inputs(c), c["cu"].cuda(), s, state_out=s, gate=gate)
        assert l3 is s and torch.equal(y3, y) and torch.equal(s, last), "in place"


@pytest.mark.parametrize("lam,g,z,gate", FORMS)
@pytest.mark.parametrize("rows,d,io", [(1, 1, "f32"), (3, 65, "bf16"), (257, 40, "f32"), (5, 1026, "bf16")])
def test_decode(rows, d, io, lam, g, z, gate):
    c = ref.gated_inputs(2, [1] * rows, d, io, lam, g, z)
    s = c["state"].cuda()
    y, last = mm.gated_decode(*strided(c), s, gate=gate)
    want, wl, mag, lmag, _ = ref.gated(c, gate)
    ref.check(y, want, mag, 1, "y")
    ref.check(last, wl, lmag, 1, "state")
    y2, s2 = mm.gated_decode(*inputs(c), s, state_out=s, gate=gate)
    assert s2 is s and torch.equal(y2, y) and torch.equal(s, last)
    c["state"] = None
    y, last = mm.gated_decode(*inputs(c), gate=gate)
    want, wl, mag, lmag, _ = ref.gated(c, gate)
    ref.check(y, want, mag, 1, "y from zeros")
    ref.check(last, wl, lmag, 1, "state from zeros")


@pytest.mark.parametrize("lam,g,z,gate", FORMS)
@pytest.mark.parametrize("lens,d,io", CASES)
def test_backward(lens, d, io, lam, g, z, gate):
    plain = z and not lam
    c = ref.gated_inputs(3, lens, d, io, lam, g, z, state=not plain)
    T = sum(lens)
    want = ref.gated_backward(c, gate, dstate=not plain)
    ds = None if plain else c["dstate"].cuda()
    both = torch.full((T, 4 * d + 1), ref.NAN, dtype=c["x"].dtype, device="cuda")
    given = {n: both[:, i * d:(i + 1) * d] for i, n in enumerate(("dx", "dr", "dg", "dz")) if c[n[1:]] is not None}
    got = mm.gated_backward(*strided(c), c["cu"].cuda(), gpu(c["state"]), c["dy"].cuda(), ds, gate=gate, **given)
    assert both[:, 4 * d].isnan().all()
    for k, (v, mag) in want.items():
        ref.check(got[k], v, mag, T, k)
    assert {k for k, v in got.items() if v is not None} == set(want)
    _, _, ckpt = mm.gated_prefill_train(*inputs(c), c["cu"].cuda(), gpu(c["state"]), gate=gate)
    kept = mm.gated_backward(*inputs(c), c["cu"].cuda(), gpu(c["state"]), c["dy"].cuda(), ds, ckpt=ckpt, gate=gate)
    for k in want:
        assert torch.equal(kept[k], got[k]), f"{k}: with the forward's checkpoints"


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_open_and_closed_gates(io):
    """Decays of exactly 1 and 0: r far out on both sides, infinities among them; lam of either end."""
    lens, d = [40, 300], 33
    c = ref.gated_inputs(4, lens, d, io, z=False)
    r = c["r"].clone()
    r[::3] = -200.0
    r[1::5] = 200.0
    r[7] = -float("inf")
    r[9] = float("inf")
    c["r"] = r
    c["lam"][0], c["lam"][1], c["lam"][2] = -200.0, 50.0, -30.0
    y, last = mm.gated_prefill(*inputs(c), c["cu"].cuda(), c["state"].cuda())
    want, wl, mag, lmag, _ = ref.gated(c)
    ref.check(y, want, mag, sum(lens), "y")
    ref.check(last, wl, lmag, sum(lens), "state")
    got = mm.gated_backward(*inputs(c), c["cu"].cuda(), c["state"].cuda(), c["dy"].cuda(), c["dstate"].cuda())
    for k, (v, m) in ref.gated_backward(c).items():
        ref.check(got[k], v, m, sum(lens), k)


@pytest.mark.parametrize("lens", [[20, 600, 5], [3, 9000, 30]])
@pytest.mark.parametrize("key,value", [("x", ref.NAN), ("r", ref.NAN), ("g", ref.NAN), ("x", float("inf")), ("state", ref.NAN)])
def test_values_that_are_not_finite_stay_in_their_sequence_and_channel(lens, key, value):
    d, hit = 70, 5
    c = ref.gated_inputs(5, lens, d, "f32", z=False)
    run = lambda k: mm.gated_prefill(*inputs(k), k["cu"].cuda(), k["state"].cuda())  # noqa: E731
    back = lambda k: mm.gated_backward(*inputs(k), k["cu"].cuda(), k["state"].cuda(), k["dy"].cuda(), k["dstate"].cuda())  # noqa: E731
    clean, cl = run(c)
    base = back(c)
    at, (lo, hi) = lens[0] + 300, (lens[0], lens[0] + lens[1])
    bad = dict(c, **{key: c[key].clone()})
    if key == "state":
        at = lo
        bad["state"][1, hit] = value
    else:
        bad[key][at, hit] = value
    y, last = run(bad)
    touched = torch.zeros_like(clean, dtype=torch.bool)
    touched[at:hi, hit] = True
    assert torch.equal(y[~touched], clean[~touched])
    assert not y[at, hit].isfinite() and not last[1, hit].isfinite()
    last[1, hit] = cl[1, hit]
    assert torch.equal(last, cl)
    got = back(bad)
    rest = [k for k in range(d) if k != hit]
    for k in ("dx", "dr", "dg"):
        assert torch.equal(got[k][:, rest], base[k][:, rest]), k
        assert torch.equal(got[k][:lo], base[k][:lo]) and torch.equal(got[k][hi:], base[k][hi:]), k
    assert torch.equal(got["dlam"][rest], base["dlam"][rest])
    up = dict(c, dy=c["dy"].clone())
    up["dy"][at, hit] = ref.NAN
    got = back(up)
    touched = torch.zeros_like(clean, dtype=torch.bool)
    touched[lo:at + 1, hit] = True
    for k in ("dx", "dr", "dg"):
        assert torch.equal(got[k][~touched], base[k][~touched]), k
        assert got[k][touched].isnan().all(), k


def test_a_nan_lam_shows():
    c = ref.gated_inputs(6, [30], 40, "bf16")
    c["lam"][3] = ref.NAN
    y, last = mm.gated_prefill(*inputs(c), c["cu"].cuda())
    assert y[:, 3].isnan().all() and y[:, 4:].isfinite().all() and last[0, 3].isnan()
    got = mm.gated_backward(*inputs(c), c["cu"].cuda(), None, c["dy"].cuda())
    assert got["dlam"][3].isnan() and got["dlam"][4:].isfinite().all()


def test_empty_calls():
    x = torch.zeros(0, 8, device="cuda", dtype=torch.bfloat16)
    lam, s = torch.ones(8, device="cuda"), torch.randn(2, 8, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    y, last, ckpt = mm.gated_prefill_train(x, x, None, None, lam, cu, s)
    assert y.shape == ckpt.shape == (0, 8) and torch.equal(last, s)
    assert not mm.gated_prefill(x, x, None, None, lam, cu)[1].any()
    g = mm.gated_backward(x, x, None, None, lam, cu, s, x, s)
    assert torch.equal(g["dstate_in"], s) and not g["dlam"].any()
