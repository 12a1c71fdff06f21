"""The causal convolution by itself against its definition in 64 bits.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

# lens, d, W, io: empty and short sequences, sequences that start and end anywhere in a tile, odd channels, several tiles
CASES = [([1], 1, 4, "f32"), ([1, 0, 2, 3, 1], 5, 4, "bf16"), ([4, 300, 0, 17], 64, 4, "bf16"), ([16, 16, 32], 70, 3, "f32"),
         ([100], 33, 2, "bf16"), ([700, 1, 2, 37], 257, 4, "f32"), ([1] * 70, 40, 3, "bf16"), ([513], 520, 4, "bf16"),
         ([15, 17, 1, 31, 64, 3], 8, 4, "bf16"), ([0, 0, 5, 0], 12, 2, "f32"), ([1100, 900], 1030, 4, "bf16"), ([0, 0], 8, 4, "f32")]


def gpu(t):
    return t.cuda() if t is not None else None


def wide(t):
    """On the GPU, still a column range of a wider tensor."""
    out = torch.zeros(t.shape[0], t.shape[1] + 3, dtype=t.dtype, device="cuda")
    out[:, 3:] = t.cuda()
    return out[:, 3:]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("bias,state", [(True, True), (False, False)])
@pytest.mark.parametrize("lens,d,W,io", CASES)
def test_prefill(lens, d, W, io, bias, state, silu):
    c = ref.conv_inputs(1, lens, d, W, io, bias, state)
    x, s0 = wide(c["x"]), gpu(c["state"])
    y, last = mm.conv_prefill(x, c["weight"].cuda(), gpu(c["bias"]), c["cu"].cuda(), s0, silu=silu)
    want, wl, mag = ref.conv(c, silu)
    ref.check(y, want, mag, W, "y")
    assert torch.equal(last.cpu().double(), wl), "the final state holds raw inputs"
    if state:
        y2, l2 = mm.conv_prefill(x, c["weight"].cuda(), gpu(c["bias"]), c["cu"].cuda(), s0, state_out=s0, silu=silu)
        assert l2 is s0 and torch.equal(y2, y) and torch.equal(s0, last), "in place"


@pytest.mark.parametrize("W,io", [(4, "bf16"), (3, "f32"), (2, "bf16")])
def test_decode_continues_a_prefill(W, io):
    c = ref.conv_inputs(2, [9, 9, 9], 65, W, io)
    x, w, b = c["x"].cuda(), c["weight"].cuda(), c["bias"].cuda()
    y, last = mm.conv_prefill(x, w, b, c["cu"].cuda(), c["state"].cuda())
    s = c["state"].cuda()
    for t in range(9):
        yt, s2 = mm.conv_decode(x[t::9], w, b, s, state_out=s)
        assert s2 is s and torch.equal(yt, y[t::9]), t
    assert torch.equal(s, last)
    y0, s0 = mm.conv_decode(x[:3], w, None, silu=False)
    assert torch.equal(s0[:, :, -1], x[:3].float()) and not s0[:, :, :-1].any()


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("bias,state", [(True, True), (False, False)])
@pytest.mark.parametrize("lens,d,W,io", CASES)
def test_backward(lens, d, W, io, bias, state, silu):
    c = ref.conv_inputs(3, lens, d, W, io, bias, state)
    want = ref.conv_backward(c, silu, dstate=state)
    both = torch.full((sum(lens), d + 7), ref.NAN, dtype=c["x"].dtype, device="cuda")
    got = mm.conv_backward(wide(c["x"]), c["weight"].cuda(), gpu(c["bias"]), c["cu"].cuda(), gpu(c["state"]), c["dy"].cuda(),
                           c["dstate"].cuda() if state else None, silu=silu, dx=both[:, 7:])
    assert (got["dbias"] is None) == (not bias) and both[:, :7].isnan().all()
    for k, (v, mag) in want.items():
        ref.check(got[k], v, mag, W if k in ("dx", "dstate_in") else sum(lens), k)
    again = mm.conv_backward(wide(c["x"]), c["weight"].cuda(), gpu(c["bias"]), c["cu"].cuda(), gpu(c["state"]), c["dy"].cuda(),
                             c["dstate"].cuda() if state else None, silu=silu, need_dstate=False)
    assert again["dstate_in"] is None
    assert all(torch.equal(again[k], got[k]) for k in want if k != "dstate_in"), "a call repeats bit for bit"


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_values_that_are_not_finite_stay_with_their_windows(io):
    lens, d, W = [20, 40, 5], 70, 4
    c = ref.conv_inputs(4, lens, d, W, io)
    clean, _ = mm.conv_prefill(c["x"].cuda(), c["weight"].cuda(), c["bias"].cuda(), c["cu"].cuda(), c["state"].cuda())
    for at, v in ((19, ref.NAN), (25, float("inf")), (59, ref.NAN)):
        x = c["x"].clone()
        x[at, 3] = v
        y, last = mm.conv_prefill(x.cuda(), c["weight"].cuda(), c["bias"].cuda(), c["cu"].cuda(), c["state"].cuda())
        end = next(hi for _, lo, hi in ref.ranges(lens) if lo <= at < hi)
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[at:min(at + W, end), 3] = True
        assert torch.equal(y[~hit], clean[~hit])
        if v != v:
            assert y[hit].isnan().all()
        dy = c["dy"].clone()
        dy[at, 3] = ref.NAN
        run = lambda g: mm.conv_backward(c["x"].cuda(), c["weight"].cuda(), c["bias"].cuda(), c["cu"].cuda(), c["state"].cuda(), g.cuda())  # noqa: E731
        got, base = run(dy), run(c["dy"])
        lo = next(lo for _, lo, hi in ref.ranges(lens) if lo <= at < hi)
        hit = torch.zeros_like(clean, dtype=torch.bool)
        hit[max(at - W + 1, lo):at + 1, 3] = True
        assert got["dx"][hit].isnan().all() and torch.equal(got["dx"][~hit], base["dx"][~hit])
        rest = [k for k in range(d) if k != 3]
        assert got["dbias"][3].isnan() and torch.equal(got["dbias"][rest], base["dbias"][rest])


def test_empty_calls():
    x = torch.zeros(0, 8, device="cuda", dtype=torch.bfloat16)
    w, s = torch.ones(8, 4, device="cuda"), torch.randn(2, 8, 3, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    y, last = mm.conv_prefill(x, w, None, cu, s)
    assert y.shape == (0, 8) and torch.equal(last, s)
    g = mm.conv_backward(x, w, w[:, 0].contiguous(), cu, s, x, s)
    assert torch.equal(g["dstate_in"], s) and not g["dweight"].any() and not g["dbias"].any()


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_long_walks(io):
    """Enough tokens for walks of 64: sequences that start and end at every place of them, and sequences of many walks."""
    lens = [61, 3, 64, 1, 127, 2, 0, 66, 4000, 62, 65, 130, 1, 1, 1, 7000] + [37] * 70
    c = ref.conv_inputs(5, lens, 1028, 4, io)
    x, w, b, cu, s0 = wide(c["x"]), c["weight"].cuda(), c["bias"].cuda(), c["cu"].cuda(), c["state"].cuda()
    y, last = mm.conv_prefill(x, w, b, cu, s0)
    want, wl, mag = ref.conv(c, True)
    ref.check(y, want, mag, 4, "y")
    assert torch.equal(last.cpu().double(), wl)
    got = mm.conv_backward(x, w, b, cu, s0, c["dy"].cuda(), c["dstate"].cuda())
    for k, (v, m) in ref.conv_backward(c, True).items():
        ref.check(got[k], v, m, 4 if k in ("dx", "dstate_in") else sum(lens), k)
