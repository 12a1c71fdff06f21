"""Calls on a stream that is behind the current one: memory that the call allocated must not go to the current
stream's next allocations before the call is done with it.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import heads_ref as ref
from tests.test_gpu_heads import to_gpu, tokens

pytestmark = pytest.mark.gpu


def heads(op):
    g = to_gpu(ref.heads_inputs(41, [900, 400], 4, 64, 2, 128, "bf16"))
    if op == "prefill":
        return lambda **kw: mm.heads_prefill(*tokens(g), g["cu"], g["state"], **kw)
    return lambda **kw: list(mm.heads_backward(*tokens(g), g["cu"], g["state"], g["dy"], g["dstate"], **kw).values())


def norm(op):
    gen = torch.Generator(device="cuda").manual_seed(42)
    y, z, do = (torch.randn(900, 1024, generator=gen, device="cuda").bfloat16() for _ in range(3))
    w = torch.randn(1024, generator=gen, device="cuda")
    if op == "gate_norm_backward":
        return lambda **kw: mm.gate_norm_backward(do, y, z, w, **kw)
    return lambda **kw: list(mm.residual_norm_backward(do, None, y, z, w, w, scale_vec=w, **kw).values())


def behind(stream):
    """Work that keeps the stream busy while the host goes on."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


def check(call):
    want = [t.clone() for t in call() if t is not None]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    behind(side)
    got = [t for t in call(stream=side) if t is not None]
    # the current stream's next allocations, of every size the call may have dropped
    filled = [torch.full((1 << k,), float("nan"), device="cuda") for k in range(6, 26)]
    torch.cuda.current_stream().wait_stream(side)
    copies = [t.clone() for t in got]
    del got, filled
    # dropped outputs, still read by the copies above, on the side stream's next call
    again = [t for t in call(stream=side) if t is not None]
    torch.cuda.synchronize()
    for w, c, a in zip(want, copies, again):
        assert torch.equal(w, c) and torch.equal(w, a)


@pytest.mark.parametrize("op", ["prefill", "backward"])
def test_heads_behind_the_current_stream(op):
    check(heads(op))


@pytest.mark.parametrize("op", ["gate_norm_backward", "residual_norm_backward"])
def test_norms_behind_the_current_stream(op):
    check(norm(op))
