"""Batches of many sequences through the matrix-core prefill: whether whole sequences or stretches of equal length run
is decided on the device, by the longest sequence.  Both outcomes against 64 bits, in place too, and repeated."""
import pytest
import torch

from tests import heads_ref as ref
import selective_state_space_causal_amd as mm

pytestmark = pytest.mark.gpu

BATCHES = {
    "even": [20] * 60 + [0, 1, 64, 33],
    "one long among short": [5] * 30 + [900] + [5] * 30 + [0] * 3,
    "just short of two stretches": [3] * 63 + [256],
    "just past two stretches": [3] * 63 + [257],
}


@pytest.mark.parametrize("name", BATCHES)
@pytest.mark.parametrize("N", [32, 100])
def test_prefill_of_many_sequences(name, N):
    lens = BATCHES[name]
    c = ref.heads_inputs(21, lens, 16, 64, 8, N, "bf16")
    yr, sr, ya, sa = ref.forward(c)
    g = {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}
    ref.split(g)
    args = [g[k] for k in ("x", "dt", "B", "C", "A_log", "D", "dt_bias")]
    y, s = mm.heads_prefill(*args, g["cu"], g["state"])
    torch.cuda.synchronize()
    T = sum(lens)
    ref.check(y, yr, ya, T, "y")
    ref.check(s, sr, sa, T, "state")
    st = g["state"].clone()
    y2, s2 = mm.heads_prefill(*args, g["cu"], st, state_out=st)
    assert s2 is st and torch.equal(y, y2) and torch.equal(s, st)
