"""The gated recurrence over many slots of which most have no token: their states and gradients, and that they are copied side by
side.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

# lens, d, io: empty slots before, between and behind tokens, in every place of 64, and more of them than a tile has waves for
CASES = [([0] * 700 + [3, 0, 0, 130] + [0] * 901, 66, "bf16"), ([0, 1] * 400 + [0] * 63, 5, "f32"), ([0] * 129, 200, "bf16"),
         ([0] * 63 + [5] + [0] * 64 + [1], 260, "bf16"), ([0] * 2100 + [70], 64, "f32"), ([0], 1, "f32")]


@pytest.mark.parametrize("lens,d,io", CASES, ids=[f"{len(c[0])} slots" for c in CASES])
def test_values(lens, d, io):
    c = ref.gated_inputs(8, lens, d, io)
    T = sum(lens)
    ins = [c[k].cuda() for k in ("x", "r", "g", "z", "lam", "cu", "state")]
    want, wl, mag, lmag, before = ref.gated(c)
    for state in (ins[6], None):
        if state is None:
            want, wl, mag, lmag, before = ref.gated(dict(c, state=None))
        held = torch.full((len(lens), d), ref.NAN, device="cuda")
        y, last, ckpt = mm.gated_prefill_train(*ins[:6], state, state_out=held)
        assert last is held
        ref.check(y, want, mag, T, "y")
        ref.check(last, wl, lmag, T, "state")
        ref.check(ckpt, *(t[::mm.layer.GATED_BLOCK] for t in before), T, "checkpoints")
        empty = torch.tensor(lens) == 0
        assert torch.equal(last[empty.cuda()].cpu(), c["state"][empty] if state is not None else torch.zeros(int(empty.sum()), d))
        s = torch.zeros_like(held) if state is None else state.clone()
        y2, s2 = mm.gated_prefill(*ins[:6], s, state_out=s)
        assert s2 is s and torch.equal(s, last) and torch.equal(y2, y), "in place"
    got = mm.gated_backward(*ins, c["dy"].cuda(), c["dstate"].cuda())
    for k, (v, m) in ref.gated_backward(c).items():
        ref.check(got[k], v, m, T, k)
    assert torch.equal(got["dstate_in"][empty.cuda()].cpu(), c["dstate"][empty])
    got = mm.gated_backward(*ins, c["dy"].cuda(), need_dstate=False)
    assert got["dstate_in"] is None
    got = mm.gated_backward(*ins, c["dy"].cuda())
    assert not got["dstate_in"][empty.cuda()].any(), "nothing asked of the final states"


def test_captured_and_on_another_stream():
    """More slots than tokens, forward and backward in one graph, replayed between eager calls; then behind the current stream."""
    from tests.test_gpu_streams import check

    lens, d = [0] * 900 + [70] + [0] * 500 + [3] + [0] * 60, 132
    c = ref.gated_inputs(9, lens, d, "bf16")
    ins = [c[k].cuda() for k in ("x", "r", "g", "z", "lam", "cu", "state")]
    dy, dstate = c["dy"].cuda(), c["dstate"].cuda()

    def both(**kw):
        return [*mm.gated_prefill(*ins, **kw), *mm.gated_backward(*ins, dy, dstate, **kw).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for i in range(4):
        ins[6].add_(0.25)
        dstate.add_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(held, both())):
            assert torch.equal(a, b), (i, j)
    check(lambda **kw: list(mm.gated_prefill(*ins, **kw)))
    check(lambda **kw: list(mm.gated_backward(*ins, dy, dstate, **kw).values()))


def test_time():
    """40000 slots, 16 tokens: about as long as the convolution takes, whose threads copy a slot and channel each."""
    S, T, d = 40000, 16, 256
    x, lam, st, w = (torch.randn(*s, device="cuda") for s in ((T, d), (d,), (S, d), (d, 2)))
    cu = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    cu[S // 2:] = T

    def microseconds(call):
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

    conv = microseconds(lambda: mm.conv_prefill(x, w, None, cu, st[..., None]))
    for name, call in (("forward", lambda: mm.gated_prefill(x, x, x, x, lam, cu, st)),
                       ("backward", lambda: mm.gated_backward(x, x, x, x, lam, cu, st, x, st))):
        us = microseconds(call)
        print(f"{name}: {us:.0f} us, convolution {conv:.0f} us")
        assert us <= 3 * conv + 100
