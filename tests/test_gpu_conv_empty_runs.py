"""The causal convolution with many empty sequences between two tokens: values, states and gradients against 64 bits, and that the
empty ones cost no chain of accesses.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

LENS = [0] * 300 + [1, 2] + [0] * 5000 + [1, 70] + [0, 3] * 50 + [0] * 3000 + [9] + [0] * 7


@pytest.mark.parametrize("d,W,io", [(5, 4, "f32"), (8, 3, "bf16"), (66, 2, "bf16")])
def test_values(d, W, io):
    c = ref.conv_inputs(6, LENS, d, W, io)
    x, w, b, cu, s0 = (c[k].cuda() for k in ("x", "weight", "bias", "cu", "state"))
    y, last = mm.conv_prefill(x, w, b, cu, s0)
    want, wl, mag = ref.conv(c, True)
    ref.check(y, want, mag, W, "y")
    assert torch.equal(last.cpu().double(), wl)
    got = mm.conv_backward(x, w, b, cu, s0, c["dy"].cuda(), c["dstate"].cuda())
    for k, (v, m) in ref.conv_backward(c, True).items():
        ref.check(got[k], v, m, W if k in ("dx", "dstate_in") else sum(LENS), k)


def test_time():
    """400000 empty sequences between two tokens take about as long as behind the last one, where no walk crosses them."""
    n, d = 400000, 4
    x, w = torch.randn(40, d, device="cuda"), torch.randn(d, 4, device="cuda")
    s0 = torch.randn(n + 2, d, 3, device="cuda")

    def microseconds(cu, backward):
        call = ((lambda: mm.conv_backward(x, w, None, cu, s0, x)) if backward else (lambda: mm.conv_prefill(x, w, None, cu, s0)))
        call()
        best = float("inf")
        for _ in range(5):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b) * 1e3)
        return best

    between = torch.cat([torch.tensor([0]), torch.full((n + 1,), 18), torch.tensor([40])]).to("cuda", torch.int32)
    behind = torch.cat([torch.tensor([0, 18]), torch.full((n + 1,), 40)]).to("cuda", torch.int32)
    for backward in (False, True):
        crossed, not_crossed = microseconds(between, backward), microseconds(behind, backward)
        print(f"{'backward' if backward else 'forward'}: {crossed:.0f} us, {not_crossed:.0f} us with none to cross")
        assert crossed <= 3 * not_crossed + 100
