"""The gated recurrence and the convolution where gates and inputs hold the type's lowest and largest values.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

LENS = [130, 1, 0, 70]


@pytest.mark.parametrize("gate", ["silu", "gelu"])
@pytest.mark.parametrize("lam", [True, False])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_gates(io, lam, gate):
    """r and g wide open and shut: decays, inputs and gradients as the formulas have them.  z at the lowest value: its token's output
    and gradients are zeros, whatever the bound says that z's size lets them be."""
    c = ref.gated_inputs(3, LENS, 66, io, lam)
    most = torch.finfo(ref.DT[io]).max
    for k, other in (("r", most), ("g", most), ("z", -most / 2)):
        t = c[k].clone()
        t[5::7], t[9::11] = -most, other
        c[k] = t
    shut = c["z"].float() < -1e30
    cuda = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    ins = [cuda[k] for k in ("x", "r", "g", "z", "lam", "cu", "state")]
    y, last = mm.gated_prefill(*ins, gate=gate)
    want, wl, mag, lmag, _ = ref.gated(c, gate)
    assert not y.cpu()[shut].any()
    ref.check(y, torch.where(shut, 0.0, want), torch.where(shut, 0.0, mag), sum(LENS), "y")
    ref.check(last, wl, lmag, sum(LENS), "state")
    got = mm.gated_backward(*ins, cuda["dy"], cuda["dstate"], gate=gate)
    # what a shut token's dy asks of the states is 0: with a dy of 0 there, the other gradients' magnitudes are as they should be
    quiet = dict(c, dy=torch.where(shut, 0.0, c["dy"].float()).to(c["dy"].dtype), z=torch.where(shut, 0.0, c["z"].float()).to(c["z"].dtype))
    exact = ref.gated_backward(quiet, gate)
    assert not got["dz"].cpu()[shut].any()
    for k, (v, m) in exact.items():
        ref.check(got[k], v, m, sum(LENS), k)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_convolution(io):
    T, d, W = 50, 64, 4
    c = ref.conv_inputs(4, [T], d, W, io, bias=False, state=False)
    c["weight"] = torch.full((d, W), 0.25)
    c["x"] = c["x"].clone()
    c["x"][7] = -torch.finfo(ref.DT[io]).max  # a quarter of it: u is finite, its sigmoid 0
    y, _ = mm.conv_prefill(c["x"].cuda(), c["weight"].cuda(), None, c["cu"].cuda())
    assert not y[7:7 + W].any() and y.isfinite().all()
    got = mm.conv_backward(c["x"].cuda(), c["weight"].cuda(), None, c["cu"].cuda(), None, c["dy"].cuda())
    assert got["dx"].isfinite().all() and not got["dx"][7].any(), "no slope where the sigmoid is 0"
