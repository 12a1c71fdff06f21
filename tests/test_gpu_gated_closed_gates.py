"""The gated recurrence where a gate is all but closed: r where 1 + exp(-r) is past the largest number whose reciprocal is
normal, with and without lam.  Needs an MI355X.

Float32 has no full precision below 2^-126, and what is there may count as 0.  Without lam that is a decay off by 2^-126 of
the state before, inside the 1e-30 of `ref.check`.  With lam all of these r have rho < 2^-124 and so 1 - a^2 = 2 c softplus(lam)
rho at 2^-126 or below (softplus(lam) < 0.014 here): m, its root, may be anything from 0 to 2^-63.  With B the
largest of the inputs and 1, |u| <= B, a state and an adjoint are at most (T + 1) B, and L / m = m / 2: each output is a sum of
at most T terms m u, G m, G m u or G u L / m (those with L itself are smaller still), so that the error is at most
2^-63 T (T + 1) B^2.
"""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

GRID = torch.arange(-90.0, -85.5, 0.5)  # every bfloat16 value of [-90, -86]
FINE = torch.linspace(-90.0, -86.0, 4001)


def gpu(t):
    return t.cuda() if t is not None else None


def inputs(c):
    return [gpu(c[k]) for k in ("x", "r", "g", "z", "lam")]


def closed(lens, d, io, lam, grid, seed=21):
    """Inputs whose r is from the grid, and what an output may be off by for m alone, as a magnitude for `ref.check`."""
    c = ref.gated_inputs(seed, lens, d, io, lam, z=False)
    pick = torch.randint(0, len(grid), c["r"].shape, generator=torch.Generator().manual_seed(seed))
    c["r"] = grid[pick].to(ref.DT[io])
    T, B = sum(lens), max(1.0, *(float(c[k].abs().max()) for k in ("x", "dy", "state", "dstate")))
    return c, 2.0 ** -63 * T * (T + 1) * B * B / (24 * 2.0 ** -23) if lam else 0.0


FORMS = [("bf16", True, GRID), ("bf16", False, GRID), ("f32", True, GRID), ("f32", False, FINE)]


@pytest.mark.parametrize("d", [33, 66, 64])
@pytest.mark.parametrize("io,lam,grid", FORMS, ids=["bf16 lam", "bf16", "f32 lam", "f32"])
def test_prefill_and_one_token(io, lam, grid, d):
    for lens in ([150, 1, 0, 300], [1] * 40):
        c, slack = closed(lens, d, io, lam, grid)
        want, wl, mag, lmag, _ = ref.gated(c)
        y, last = mm.gated_prefill(*inputs(c), c["cu"].cuda(), c["state"].cuda())
        ref.check(y, want, mag + slack, sum(lens), "y")
        ref.check(last, wl, lmag + slack, sum(lens), "state")
    y, last = mm.gated_decode(*inputs(c), c["state"].cuda())  # the forty sequences of one token
    ref.check(y, want, mag + slack, 1, "one token")
    ref.check(last, wl, lmag + slack, 1, "one token's state")


@pytest.mark.parametrize("d", [33, 66, 64])
@pytest.mark.parametrize("io,lam,grid", FORMS, ids=["bf16 lam", "bf16", "f32 lam", "f32"])
def test_backward(io, lam, grid, d):
    lens = [150, 1, 0, 300]
    c, slack = closed(lens, d, io, lam, grid)
    got = mm.gated_backward(*inputs(c), c["cu"].cuda(), c["state"].cuda(), c["dy"].cuda(), c["dstate"].cuda())
    for k, (v, m) in ref.gated_backward(c).items():
        ref.check(got[k], v, m + slack, sum(lens), k)
