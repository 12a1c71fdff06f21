"""The layer of examples/heads_block.py: the operators run together, against the same layer in 64 bits.

Bounds.  float32: each operator and product is within 2^-23 (16 + 4 sqrt(T)) of its terms' magnitudes (T = 110:
7e-6); a pass is a chain of five of them and the backward of ten, whose norms and decays amplify an input's
relative error by a few: 10 x 5 x 7e-6 = 3.5e-4 of the largest value, for the backward 7e-4.
bfloat16: five roundings of 2^-8 at most, amplified by as much and spread at random over the columns: 5 x 2^-8 =
2e-2 of the result's norm.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

HIDDEN, SIZES, LENS = 96, (6, 16, 2, 32), [37, 1, 0, 72]
F32_FORWARD, F32_BACKWARD, BF16_NORM = 3.5e-4, 7e-4, 5 * 2.0 ** -8


def block(dtype):
    from heads_block import HeadsBlock

    return HeadsBlock(HIDDEN, *SIZES, dtype=dtype, seed=3)


def inputs(dtype, res=torch.float32):
    g = torch.Generator().manual_seed(4)
    T, S = sum(LENS), len(LENS)
    cu = torch.tensor([sum(LENS[:i]) for i in range(S + 1)], dtype=torch.int32)
    return (torch.randn(T, HIDDEN, generator=g).to(dtype), torch.randn(T, HIDDEN, generator=g).to(res), cu,
            0.5 * torch.randn(S, *SIZES[:2], SIZES[3], generator=g))


def exact(p, h, r, state, eps=1e-5):
    """The layer in 64 bits, token by token; p: its parameters by name."""
    H, P, G, N = SIZES
    d = H * P
    norm = lambda v: v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps)  # noqa: E731
    r = r + h
    u = norm(r) * p["norm"] @ p["w_in"]
    z, x, B, C, dt = u.split([d, d, G * N, G * N, H], 1)
    x, hg = x.unflatten(1, (H, P)), H // G
    B, C = (t.unflatten(1, (G, N)).repeat_interleave(hg, 1) for t in (B, C))
    delta = torch.nn.functional.softplus(dt + p["dt_bias"], threshold=700)
    a = torch.exp(-torch.exp(p["A_log"]) * delta)
    y, states, t = [], [], 0
    for s, n in enumerate(LENS):
        st = state[s]
        for _ in range(n):
            st = a[t][:, None, None] * st + (delta[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
            y.append((st * C[t][:, None, :]).sum(-1) + p["D"][:, None] * x[t])
            t += 1
        states.append(st)
    g = torch.stack(y).flatten(1) * torch.nn.functional.silu(z)
    g = norm(g.unflatten(1, (G, d // G))).flatten(1) * p["gate"]
    return g @ p["w_out"], r, torch.stack(states)


NAMES = ("w_in", "w_out", "norm", "gate", "A_log", "D", "dt_bias")


def close(got, want, tol, what):
    err = (got.double().cpu() - want).abs().max().item()
    assert err <= tol * want.abs().max().item(), (what, err, want.abs().max().item())


def test_prefill_and_gradients_in_float32():
    b = block(torch.float32)
    h, r, cu, state = inputs(torch.float32)
    p = {k: getattr(b, k).double().cpu().requires_grad_() for k in NAMES}
    leaves = [t.double().requires_grad_() for t in (h, r, state)]
    want = exact(p, *leaves)
    out, res, st, kept = b.prefill(h.cuda(), r.cuda(), cu.cuda(), state.cuda())
    for g, w, n in zip((out, res, st), want, ("out", "residual", "state")):
        close(g, w.detach(), F32_FORWARD, n)
    gen = torch.Generator().manual_seed(5)
    up = [torch.randn(w.shape, generator=gen) for w in want]
    torch.autograd.backward(want, [u.double() for u in up])
    got = b.backward(kept, *(u.cuda() for u in up))
    for n in NAMES:
        close(got[n], p[n].grad, F32_BACKWARD, n)
    for n, leaf in zip(("h", "residual", "state"), leaves):
        close(got[n], leaf.grad, F32_BACKWARD, n)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_steps_continue_a_prefill(dtype):
    """The last tokens of the last sequence taken one at a time, from the state the others left."""
    b = block(dtype)
    h, r, cu, state = (t.cuda() for t in inputs(dtype))
    whole, res, want, _ = b.prefill(h, r, cu, state)
    k = 5
    T = sum(LENS)
    cut = cu.clone()
    cut[-1] -= k
    _, _, st, _ = b.prefill(h[:T - k], r[:T - k], cut, state)
    st = st[-1:].clone()
    for t in range(T - k, T):
        row = r[t:t + 1].clone()
        out = b.step(h[t:t + 1], row, st)
        if dtype == torch.float32:
            close(out, whole[t:t + 1].double().cpu(), 2 * F32_FORWARD, "out")
            close(row, res[t:t + 1].double().cpu(), 2 * F32_FORWARD, "residual")
        else:
            w = whole[t:t + 1].double()
            assert (out.double() - w).norm() <= 2 * BF16_NORM * w.norm()
    if dtype == torch.float32:
        close(st, want[-1:].double().cpu(), 2 * F32_FORWARD, "state")
    else:
        assert (st - want[-1:]).norm() <= 2 * BF16_NORM * want[-1:].norm()


def test_a_captured_step_replays_as_the_eager_one():
    b = block(torch.bfloat16)
    Bs = 3
    g = torch.Generator().manual_seed(6)
    h = torch.randn(Bs, HIDDEN, generator=g).to("cuda", torch.bfloat16)
    r0 = torch.randn(Bs, HIDDEN, generator=g).cuda()
    s0 = torch.randn(Bs, *SIZES[:2], SIZES[3], generator=g).cuda()
    r, s = r0.clone(), s0.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(h, r, s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step(h, r, s)
    r.copy_(r0)
    s.copy_(s0)
    er, es = r0.clone(), s0.clone()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        want = b.step(h, er, es)
        assert torch.equal(out, want) and torch.equal(r, er) and torch.equal(s, es)
        (want.float() @ want.float().t()).sum().item()  # other work between the replays
