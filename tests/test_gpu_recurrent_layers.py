"""The layers of examples/recurrent_layers.py: the convolution, the gated recurrence, the head norm and the head scan run
together, against the same layers in 64 bits.  Needs an MI355X.

Bounds.  float32: each operator and product is within 2^-23 (24 + 4 sqrt(T)) of its terms' magnitudes (T = 110: 8e-6); a pass is
a chain of seven of them and the backward of fourteen, whose norms and decays amplify an input's relative error by a few:
10 x 7 x 8e-6 = 5.6e-4 of the largest value, for the backward 1.2e-3.
bfloat16: seven roundings of 2^-8 at most, amplified by as much and spread at random over the columns: 7 x 2^-8 = 2.8e-2 of the
result's norm.
"""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from tests import layer_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

HIDDEN, LENS = 96, [37, 1, 0, 72]
F32_FORWARD, F32_BACKWARD, BF16_NORM = 5.6e-4, 1.2e-3, 7 * 2.0 ** -8
KINDS = ["gated", "retention"]


def layer(kind, dtype):
    import recurrent_layers as ex

    return ex.GatedLayer(HIDDEN, 80, dtype, seed=3) if kind == "gated" else ex.RetentionLayer(HIDDEN, 6, 16, 2, 32, dtype, seed=3)


def inputs(b, dtype):
    r, T, S = ref.gen(4), sum(LENS), len(LENS)
    pos = torch.cat([torch.arange(n) + 50 * i for i, n in enumerate(LENS)]).to(torch.int32)
    return r(T, HIDDEN).to(dtype), r(T, HIDDEN), ref.cu_of(LENS), tuple(0.5 * r(*s.shape) for s in b.state(S, "cpu")), pos


def norm(v, w, eps=1e-5):
    return v * torch.rsqrt(v.square().mean(-1, keepdim=True) + eps) * w


def exact(kind, b, p, h, r, conv_state, state, pos):
    """The layer in 64 bits, token by token; p: its parameters by name."""
    r = r + h
    proj = norm(r, p["norm"]) @ p["w_in"]
    if kind == "gated":
        d = b.d
        c = dict(lens=LENS, W=4)
        u, conv, _ = ref.conv(c, False, [proj[:, :d], p["conv_w"], p["conv_b"], conv_state])
        gates = u @ p["w_gates"]
        y, last = ref.gated(c, "gelu", [u, gates[:, :d], gates[:, d:], proj[:, d:], p["lam"], state])[:2]
        return y @ p["w_out"], r, conv, last
    H, P, G, N = b.sizes
    d = H * P
    u, conv, _ = ref.conv(dict(lens=LENS, W=4), True, [proj[:, d:], p["conv_w"], p["conv_b"], conv_state])
    x, B, C = u.split([d, G * N, G * N], 1)
    x, B, C = x.unflatten(1, (H, P)), B.unflatten(1, (G, N)), C.unflatten(1, (G, N))
    f = pos.double()[:, None, None] * b.freq.double().cpu()

    def turn(v):
        i, j = v[..., :N // 2], v[..., N // 2:]
        return torch.cat([i * torch.cos(f) - j * torch.sin(f), j * torch.cos(f) + i * torch.sin(f)], -1)

    q, k = (turn(norm(v, w)).repeat_interleave(H // G, 1) for v, w in ((C, p["q_norm"]), (B, p["k_norm"])))
    a = torch.exp(-torch.exp(p["A_log"]))[:, None, None]
    ys, lasts = [], []
    for s, lo, hi in ref.ranges(LENS):
        st = state[s]
        for t in range(lo, hi):
            st = a * st + x[t][:, :, None] * k[t][:, None, :]
            ys.append((st * q[t][:, None, :]).sum(-1))
        lasts.append(st)
    y = torch.stack(ys).flatten(1) * torch.nn.functional.silu(proj[:, :d])
    y = norm(y.unflatten(1, (G, d // G)), 1.0).flatten(1) * p["gate"]
    return y @ p["w_out"], r, conv, torch.stack(lasts)


def close(got, want, tol, what):
    err = (got.double().cpu() - want).abs().max().item()
    assert err <= tol * want.abs().max().item(), (what, err, want.abs().max().item())


def on_gpu(h, r, cu, state, pos):
    return h.cuda(), r.cuda(), cu.cuda(), tuple(s.cuda() for s in state), pos.cuda()


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_and_gradients_in_float32(kind):
    b = layer(kind, torch.float32)
    h, r, cu, state, pos = inputs(b, torch.float32)
    p = {k: getattr(b, k).double().cpu().requires_grad_() for k in b.names}
    leaves = [t.double().requires_grad_() for t in (h, r, *state)]
    want = exact(kind, b, p, *leaves, pos)
    out, res, st, kept = b.prefill(*on_gpu(h, r, cu, state, pos))
    for g, w, n in zip((out, res, *st), want, ("out", "residual", "conv state", "state")):
        close(g, w.detach(), F32_FORWARD, n)
    rnd = ref.gen(5)
    up = [rnd(*w.shape) for w in want]
    torch.autograd.backward(want, [u.double() for u in up])
    got = b.backward(kept, up[0].cuda(), up[1].cuda(), tuple(u.cuda() for u in up[2:]))
    for n in b.names:
        close(got[n], p[n].grad, F32_BACKWARD, n)
    for g, leaf, n in zip((got["h"], got["residual"], *got["state"]), leaves, ("h", "residual", "conv state", "state")):
        close(g, leaf.grad, F32_BACKWARD, n)


@pytest.mark.parametrize("kind", KINDS)
def test_prefill_in_bfloat16(kind):
    b = layer(kind, torch.bfloat16)
    h, r, cu, state, pos = inputs(b, torch.bfloat16)
    p = {k: getattr(b, k).double().cpu() for k in b.names}
    want = exact(kind, b, p, h.double(), r.double(), *(s.double() for s in state), pos)
    out, res, st, _ = b.prefill(*on_gpu(h, r, cu, state, pos))
    for g, w, n in zip((out, *st), (want[0], *want[2:]), ("out", "conv state", "state")):
        assert (g.double().cpu() - w).norm() <= BF16_NORM * w.norm(), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", KINDS)
def test_steps_continue_a_prefill(kind, dtype):
    """The last tokens of the last sequence taken one at a time, from the states the others left."""
    b = layer(kind, dtype)
    h, r, cu, state, pos = on_gpu(*inputs(b, dtype))
    whole, res, want, _ = b.prefill(h, r, cu, state, pos)
    k, T = 5, sum(LENS)
    cut = cu.clone()
    cut[-1] -= k
    _, _, st, _ = b.prefill(h[:T - k], r[:T - k], cut, state, pos[:T - k].contiguous())
    st = tuple(s[-1:].clone() for s in st)
    for t in range(T - k, T):
        row = r[t:t + 1].clone()
        out = b.step(h[t:t + 1], row, st, pos[t:t + 1].contiguous())
        w = whole[t:t + 1].double()
        if dtype == torch.float32:
            close(out, w.cpu(), 2 * F32_FORWARD, "out")
            close(row, res[t:t + 1].double().cpu(), 2 * F32_FORWARD, "residual")
        else:
            assert (out.double() - w).norm() <= 2 * BF16_NORM * w.norm()
    for g, w in zip(st, want):
        assert (g.double() - w[-1:].double()).norm() <= 2 * (F32_FORWARD if dtype == torch.float32 else BF16_NORM) * w[-1:].double().norm()


@pytest.mark.parametrize("kind", KINDS)
def test_captured_steps_and_prefills_replay_as_the_eager_ones(kind):
    b = layer(kind, torch.bfloat16)
    rnd, Bs = ref.gen(6), 3
    h, r0 = rnd(Bs, HIDDEN).to("cuda", torch.bfloat16), rnd(Bs, HIDDEN).cuda()
    s0 = tuple(rnd(*s.shape).cuda() for s in b.state(Bs, "cpu"))
    pos = torch.tensor([3, 700, 12345], dtype=torch.int32, device="cuda")
    r, s = r0.clone(), tuple(t.clone() for t in s0)
    ph, pr, cu, state, ppos = on_gpu(*inputs(b, torch.bfloat16))
    g = rnd(sum(LENS), HIDDEN).to("cuda", torch.bfloat16)

    def train():
        out, res, st, kept = b.prefill(ph, pr, cu, state, ppos)
        got = b.backward(kept, g, None)
        return [out, *st, got["h"], got["residual"], *got["state"]] + [got[n] for n in b.names]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(h, r, s, pos)
        train()
    torch.cuda.current_stream().wait_stream(side)
    steps, passes = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(steps):
        out = b.step(h, r, s, pos)
    with torch.cuda.graph(passes):
        held = train()
    r.copy_(r0)
    for t, t0 in zip(s, s0):
        t.copy_(t0)
    er, es = r0.clone(), tuple(t.clone() for t in s0)
    for i in range(4):
        steps.replay()
        torch.cuda.synchronize()
        want = b.step(h, er, es, pos)
        assert torch.equal(out, want) and torch.equal(r, er) and all(torch.equal(a, c) for a, c in zip(s, es))
        ph.copy_(ph + 0.125)
        passes.replay()
        torch.cuda.synchronize()
        for j, (a, c) in enumerate(zip(held, train())):
            assert torch.equal(a, c), (i, j)
        (want.float() @ want.float().t()).sum().item()  # other work between the replays
