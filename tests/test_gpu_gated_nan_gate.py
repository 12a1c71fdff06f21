"""A NaN in the gated recurrence's r reaches the outputs and the gradients of its own token, with and without lam.  Needs an
MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[20, 600, 5], [3, 9000, 30]], ids=str)
@pytest.mark.parametrize("io,d", [("f32", 70), ("bf16", 70), ("bf16", 72)])
@pytest.mark.parametrize("lam", [True, False])
def test_a_nan_in_r(lam, io, d, lens):
    hit, lo, hi = 5, lens[0], lens[0] + lens[1]
    at = lo + 300
    c = ref.gated_inputs(5, lens, d, io, lam, z=False)
    bad = dict(c, r=c["r"].clone())
    bad["r"][at, hit] = ref.NAN

    def run(k):
        ins = [k[n].cuda() if k[n] is not None else None for n in ("x", "r", "g", "z", "lam", "cu", "state")]
        return mm.gated_prefill(*ins)[0], mm.gated_backward(*ins, k["dy"].cuda(), k["dstate"].cuda())

    y, got = run(bad)
    clean, base = run(c)
    after = torch.zeros_like(clean, dtype=torch.bool)
    after[at:hi, hit] = True
    assert y[after].isnan().all() and torch.equal(y[~after], clean[~after])
    before = torch.zeros_like(after)
    before[lo:at + 1, hit] = True
    for k in ("dx", "dg", "dr"):  # 1 - rho is a factor of the token's own dx and dg, G of all before it
        assert got[k][before].isnan().all(), k
    same = ~before
    assert torch.equal(got["dx"][same], base["dx"][same]), "dx of later tokens does not depend on it"
    rest = ~(before | after)
    for k in ("dg", "dr"):
        assert torch.equal(got[k][rest], base[k][rest]), k
