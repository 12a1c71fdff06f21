"""NaN in what makes the decays (dt, dt_bias, A_log) shows in the results: by the formulas a NaN step or decay makes the
state NaN from its token on, in its head and sequence alone.  And decays that vanish altogether.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import heads_ref as ref
from tests.test_gpu_heads import check_prefill, run_backward, run_prefill, to_gpu, tokens
from tests.test_gpu_heads_paths import prefill_stretch

pytestmark = pytest.mark.gpu

NAN = float("nan")
# lens, H, P, G, N, io: cut and whole sequences on the matrix cores, and token by token
SHAPES = {
    "cut": ([90, 200, 40], 4, 64, 2, 128, "bf16"),
    "cut, odd": ([90, 200, 40], 6, 20, 3, 50, "bf16"),
    "whole": ([65, 200, 70] * 22, 16, 64, 8, 32, "bf16"),
    "wide": ([90, 200, 40], 2, 64, 1, 200, "bf16"),
    "float32": ([90, 200, 40], 3, 20, 1, 24, "f32"),
}


def inputs(name):
    lens, H, P, G, N, io = SHAPES[name]
    if io == "bf16" and N <= 128:
        assert prefill_stretch(lens, H, P, G)[1] == (name == "whole")
    return ref.heads_inputs(51, lens, H, P, G, N, io)


def spoiled(c, key, where):
    d = dict(c, proj=c["proj"].clone())
    ref.split(d)
    if key == "dt":
        d["dt"][where] = NAN
    else:
        d[key] = c[key].clone()
        d[key][where] = NAN
    return d


def others(n, h):
    return [i for i in range(n) if i != h]


@pytest.mark.parametrize("name", SHAPES)
def test_prefill_nan_step(name):
    c = inputs(name)
    clean_y, clean_s = run_prefill(c)
    n0, n1 = c["lens"][:2]
    h, at, hi = 1, n0 + 100, n0 + n1
    y, s = run_prefill(spoiled(c, "dt", (at, h)))
    rest = others(c["H"], h)
    assert torch.equal(y[:, rest], clean_y[:, rest]) and torch.equal(s[:, rest], clean_s[:, rest]), "other heads"
    assert torch.equal(y[:n0], clean_y[:n0]) and torch.equal(y[hi:], clean_y[hi:]), "other sequences"
    assert torch.equal(s[0], clean_s[0]) and torch.equal(s[2:], clean_s[2:])
    before = y[n0:at].float() - clean_y[n0:at].float()
    assert before.abs().max() <= 0.02 * clean_y.float().abs().max(), "earlier tokens"
    assert torch.isnan(y[at:hi, h]).all() and torch.isnan(s[1, h]).all()


@pytest.mark.parametrize("key", ["A_log", "dt_bias"])
@pytest.mark.parametrize("name", SHAPES)
def test_prefill_nan_parameter(name, key):
    c = inputs(name)
    clean_y, clean_s = run_prefill(c)
    y, s = run_prefill(spoiled(c, key, 1))
    rest = others(c["H"], 1)
    assert torch.equal(y[:, rest], clean_y[:, rest]) and torch.equal(s[:, rest], clean_s[:, rest])
    assert torch.isnan(y[:, 1]).all() and torch.isnan(s[:, 1]).all()


@pytest.mark.parametrize("key", ["dt", "A_log", "dt_bias"])
@pytest.mark.parametrize("N,io", [(128, "bf16"), (50, "bf16"), (24, "f32")])
def test_decode_nan(N, io, key):
    c = ref.heads_inputs(52, [1] * 3, 4, 20, 2, N, io)
    g = to_gpu(c)
    clean_y, clean_s = mm.heads_decode(*tokens(g), g["state"])
    g = to_gpu(spoiled(c, key, (1, 2) if key == "dt" else 2))
    y, s = mm.heads_decode(*tokens(g), g["state"])
    nan = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    nan[(1, 2) if key == "dt" else (slice(None), 2)] = True
    assert torch.isnan(y[nan]).all() and torch.isnan(s[nan]).all()
    assert torch.equal(y[~nan], clean_y[~nan]) and torch.equal(s[~nan], clean_s[~nan])


BACKWARD = [([90, 200, 40], 4, 64, 2, 128, "bf16"), ([90, 200, 40], 6, 20, 3, 50, "bf16"), ([90, 200, 40], 2, 64, 1, 200, "bf16"),
            ([90, 200, 40], 3, 20, 1, 24, "f32")]


@pytest.mark.parametrize("shape", BACKWARD)
def test_backward_nan_step(shape):
    lens, H, P, G, N, io = shape
    c = ref.heads_inputs(53, lens, H, P, G, N, io)
    clean = run_backward(c)
    n0, at, h = 90, 190, 1
    got = run_backward(spoiled(c, "dt", (at, h)))
    rest = others(H, h)
    for k in ("dx", "ddt"):
        assert torch.equal(got[k][:, rest], clean[k][:, rest]), f"{k}: other heads"
        assert torch.equal(got[k][:n0], clean[k][:n0]) and torch.equal(got[k][290:], clean[k][290:]), f"{k}: other sequences"
        assert torch.isnan(got[k][n0:at + 1, h]).all(), f"{k}: up to the token"
    for k in ("dB", "dC"):
        assert torch.equal(got[k][:n0], clean[k][:n0]) and torch.equal(got[k][290:], clean[k][290:]), k
    g = h // (H // G)
    assert torch.isnan(got["dB"][n0:at + 1, g]).all() and torch.isnan(got["dC"][at:290, g]).all()
    for k in ("dA_log", "ddt_bias"):
        assert torch.isnan(got[k][h]) and torch.equal(got[k][rest], clean[k][rest]), k
    s = got["dstate_in"]
    assert torch.isnan(s[1, h]).all() and torch.equal(s[[0, 2]], clean["dstate_in"][[0, 2]])
    assert torch.equal(s[:, rest], clean["dstate_in"][:, rest])


@pytest.mark.parametrize("shape", BACKWARD)
def test_backward_nan_decay(shape):
    lens, H, P, G, N, io = shape
    c = ref.heads_inputs(54, lens, H, P, G, N, io)
    clean, got = run_backward(c), run_backward(spoiled(c, "A_log", 1))
    rest = others(H, 1)
    assert torch.isnan(got["dA_log"][1]) and torch.isnan(got["dstate_in"][:, 1]).all()
    for k in ("dA_log", "ddt_bias", "dD"):
        assert torch.equal(got[k][rest], clean[k][rest]), k
    for k in ("dx", "ddt"):
        assert torch.equal(got[k][:, rest], clean[k][:, rest]), k


@pytest.mark.parametrize("name", SHAPES)
def test_decays_that_vanish(name):
    """exp(A_log) past float32: every decay is 0, and places without a token still leave the state as it is."""
    c = inputs(name)
    c["A_log"][1] = 100.0
    check_prefill(c, *run_prefill(c))
