"""NaN and infinities in dy, x, B and C reach the gradients that depend on them and no others: those of the later (or
earlier) tokens that the causal mask leaves out keep their values.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

from tests import heads_ref as ref
from tests.test_gpu_heads import run_backward
from tests.test_gpu_heads_paths import head_shares

pytestmark = pytest.mark.gpu

LENS, AT = [90, 200, 40], 150
LO, HI = 90, 290  # the spoiled token's sequence

# the tokens of the sequence whose gradients depend on each input of the token AT
UP_TO, FROM, ONLY, NONE = range(LO, AT + 1), range(AT, HI), range(AT, AT + 1), range(0)
DEPEND = {
    "dy": dict(dx=UP_TO, dB=UP_TO, dC=ONLY, ddt=UP_TO),
    "x": dict(dx=NONE, dB=ONLY, dC=FROM, ddt=FROM),
    "B": dict(dx=ONLY, dB=NONE, dC=FROM, ddt=FROM),
    "C": dict(dx=UP_TO, dB=UP_TO, dC=NONE, ddt=UP_TO),
}
SHAPES = [(4, 64, 2, 128, "bf16"), (6, 20, 3, 50, "bf16"), (2, 80, 1, 16, "bf16"), (2, 64, 1, 200, "bf16"), (3, 20, 1, 24, "f32")]


def spoil(c, key, value, where=AT):
    d = dict(c, proj=c["proj"].clone(), dy=c["dy"].clone())
    ref.split(d)
    d[key][where] = value
    return d


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("key", DEPEND)
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(shape, key, value):
    H, P, G, N, io = shape
    c = ref.heads_inputs(61, LENS, H, P, G, N, io)
    want, clean, got = ref.backward(c), run_backward(c), run_backward(spoil(c, key, value))
    T = sum(LENS)
    for k, tokens in DEPEND[key].items():
        bad = torch.zeros(T, dtype=torch.bool)
        bad[list(tokens)] = True
        assert not torch.isfinite(got[k][bad.cuda()]).any(), f"{k}: tokens that depend on it"
        good = ~bad
        ref.check(got[k][good.cuda()], *(t[good] for t in want[k]), T, k)
        for part in (slice(0, LO), slice(HI, T)):
            assert torch.equal(got[k][part], clean[k][part]), f"{k}: other sequences"
    s = got["dstate_in"]
    assert torch.equal(s[[0, 2]], clean["dstate_in"][[0, 2]])
    if key in ("dy", "C"):
        assert not torch.isfinite(s[1]).any()
    else:
        assert torch.equal(s, clean["dstate_in"])


@pytest.mark.parametrize("key", ["dy", "B", "C"])
def test_backward_of_several_heads_a_workgroup(key):
    """One head's dy (or a group's B or C) spoiled among several heads that one workgroup takes."""
    lens, H, P, G, N = [3] * 150 + [70], 7, 64, 1, 64
    assert head_shares(lens, H, G) < H
    c = ref.heads_inputs(62, lens, H, P, G, N, "bf16")
    at, lo, T = 450 + 40, 450, 520
    d = dict(c, proj=c["proj"].clone(), dy=c["dy"].clone())
    ref.split(d)
    where = (at, 3) if key == "dy" else at
    d[key][where] = float("nan")
    want, clean, got = ref.backward(c), run_backward(c), run_backward(d)
    for k in ("dx", "ddt", "dB", "dC"):
        assert torch.equal(got[k][:lo], clean[k][:lo]), k
    if key == "dy":
        rest = [0, 1, 2, 4, 5, 6]
        assert torch.equal(got["dx"][:, rest], clean["dx"][:, rest]) and torch.equal(got["ddt"][:, rest], clean["ddt"][:, rest])
    after = slice(at + 1, T)
    if key != "B":
        for k in ("dx", "dB", "ddt"):
            ref.check(got[k][after], *(t[after] for t in want[k]), T, k)
    else:
        before = slice(lo, at)
        ref.check(got["dC"][before], *(t[before] for t in want["dC"]), T, "dC")
        ref.check(got["dB"], *want["dB"], T, "dB")
