"""The gated recurrence's kernels for two bfloat16 channels a thread (d a multiple of two, not of four): sequences that start and end
in every part of a tile, checkpoints in its middle, states in place.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref
from tests import test_gpu_gated as gated

pytestmark = pytest.mark.gpu

CASES = [([300, 5, 0, 1, 77, 64, 128], 130), ([1] * 300, 42), ([255, 1, 257, 0, 30], 66), ([64, 64, 0, 128, 1, 63, 7], 258),
         ([15, 17, 16, 1, 31, 700, 0, 2], 2), ([3, 2000, 0, 65], 38)]


@pytest.mark.parametrize("lam,g,z,gate", gated.FORMS)
@pytest.mark.parametrize("lens,d", CASES, ids=[f"{len(c[0])}x{c[1]}" for c in CASES])
def test_prefill(lens, d, lam, g, z, gate):
    gated.test_prefill(lens, d, "bf16", lam, g, z, gate)


@pytest.mark.parametrize("lam,g,z,gate", gated.FORMS)
@pytest.mark.parametrize("lens,d", CASES, ids=[f"{len(c[0])}x{c[1]}" for c in CASES])
def test_backward(lens, d, lam, g, z, gate):
    gated.test_backward(lens, d, "bf16", lam, g, z, gate)


def test_checkpoints_of_states_in_place():
    lens = [64, 128, 64, 2000, 48, 128, 0, 64, 192, 5000, 120, 65, 63, 128]
    c = ref.gated_inputs(11, lens, 522, "bf16")
    ins = [c[k].cuda() for k in ("x", "r", "g", "z", "lam", "cu")]
    state = c["state"].cuda()
    y, last, ckpt = mm.gated_prefill_train(*ins, state)
    for s, t in enumerate(c["cu"][:-1].tolist()):
        if t % mm.layer.GATED_BLOCK == 0 and lens[s] > 0:
            assert torch.equal(ckpt[t // mm.layer.GATED_BLOCK], state[s])
    for _ in range(5):
        st = state.clone()
        got = mm.gated_prefill_train(*ins, st, st)
        assert torch.equal(got[0], y) and torch.equal(st, last) and torch.equal(got[2], ckpt)
