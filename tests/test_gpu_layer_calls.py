"""The convolution's, the gated recurrence's and the head norm's calls as a program makes them: rows far apart, many and long
sequences, other streams, two calls at once, graphs that share a workspace.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref
from tests.test_gpu_streams import check

pytestmark = pytest.mark.gpu


def cuda(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


def conv_calls(lens, d, io, seed=1):
    c = cuda(ref.conv_inputs(seed, lens, d, 4, io))
    return [lambda **kw: list(mm.conv_prefill(c["x"], c["weight"], c["bias"], c["cu"], c["state"], **kw)),
            lambda **kw: list(mm.conv_backward(c["x"], c["weight"], c["bias"], c["cu"], c["state"], c["dy"], c["dstate"], **kw).values())]


def gated_calls(lens, d, io, seed=2):
    c = cuda(ref.gated_inputs(seed, lens, d, io))
    ins = [c[k] for k in ("x", "r", "g", "z", "lam", "cu", "state")]
    return [lambda **kw: list(mm.gated_prefill_train(*ins, **kw)),
            lambda **kw: list(mm.gated_backward(*ins, c["dy"], c["dstate"], **kw).values())]


def qk_calls(T, D, io, seed=3):
    c = cuda(ref.qk_inputs(seed, T, 4, 2, D, D // 2, io))
    rest = [c[k] for k in ("q", "k", "wq", "wk", "pos", "freq")]
    return [lambda **kw: list(mm.qk_norm(*rest, **kw)), lambda **kw: list(mm.qk_norm_backward(c["dq"], c["dk"], *rest, **kw))]


CALLS = {"conv": lambda: conv_calls([900, 400, 0, 7], 520, "bf16"), "gated": lambda: gated_calls([900, 3000, 0, 7], 260, "bf16"),
         "qk": lambda: qk_calls(1300, 64, "bf16"), "qk, any width": lambda: qk_calls(300, 20, "f32")}


@pytest.mark.parametrize("which", [0, 1], ids=["forward", "backward"])
@pytest.mark.parametrize("name", CALLS)
def test_behind_the_current_stream(name, which):
    check(CALLS[name]()[which])


@pytest.mark.parametrize("name", CALLS)
def test_two_calls_at_once(name):
    """The same call on two streams, each with memory of its own, while the other runs."""
    calls = CALLS[name]()
    want = [[t.clone() for t in f()] for f in calls]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [(f, [t for t in calls[f](stream=s)]) for _ in range(6) for s in streams for f in range(2)]
    torch.cuda.synchronize()
    for f, ts in got:
        for a, b in zip(ts, want[f]):
            assert torch.equal(a, b)


def test_graphs_that_share_a_workspace():
    """A forward and a backward captured with one workspace, replayed in turn with eager calls between them."""
    lib = mm.load()
    lens, d = [300, 5000, 1], 260
    T = sum(lens)
    c = cuda(ref.gated_inputs(4, lens, d, "bf16"))
    ins = [c[k] for k in ("x", "r", "g", "z", "lam", "cu", "state")]
    need = max(lib.mamba_mixer_gated_prefill_workspace_bytes(T, d), lib.mamba_mixer_gated_backward_workspace_bytes(T, d, 0))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    forward = lambda: list(mm.gated_prefill(*ins, workspace=ws))  # noqa: E731
    backward = lambda: list(mm.gated_backward(*ins, c["dy"], c["dstate"], workspace=ws).values())  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        forward(), backward()
    torch.cuda.current_stream().wait_stream(side)
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g, f in zip(graphs, (forward, backward)):
        with torch.cuda.graph(g):
            held.append(f())
    for i in range(4):
        c["x"].copy_(c["x"] + 0.125)
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for f, ts in zip((forward, backward), held):
            for a, b in zip(ts, f()):
                assert torch.equal(a, b), i
        ws.fill_(17 * i)


def far(t, stride):
    """The rows of t, `stride` elements apart."""
    out = torch.empty((t.shape[0] - 1) * stride + t[0].numel(), dtype=t.dtype, device="cuda")
    rows = torch.as_strided(out, (t.shape[0], t[0].numel()), (stride, 1))
    rows.copy_(t.reshape(t.shape[0], -1))
    return rows.view(t.shape) if t.dim() == 2 else torch.as_strided(out, t.shape, (stride, *t[0].contiguous().stride()))


def test_rows_whose_offsets_pass_32_bits():
    T, stride = 1100, 1 << 22  # 4.6 G elements, 9.2 GB of bfloat16
    c = cuda(ref.gated_inputs(5, [T - 100, 100], 64, "bf16"))
    x = far(c["x"], stride)
    ins = [c[k] for k in ("r", "g", "z", "lam", "cu", "state")]
    for a, b in zip(mm.gated_prefill(x, *ins), mm.gated_prefill(c["x"], *ins)):
        assert torch.equal(a, b)
    args = (c["dy"], c["dstate"])
    want = mm.gated_backward(c["x"], *ins, *args)
    out = far(torch.zeros_like(c["x"]), stride)
    got = mm.gated_backward(x, *ins, *args, dx=out)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    del out
    w, b = torch.randn(64, 4, device="cuda"), torch.randn(64, device="cuda")
    for p, q in zip(mm.conv_prefill(x, w, b, c["cu"]), mm.conv_prefill(c["x"], w, b, c["cu"])):
        assert torch.equal(p, q)
    q = far(c["x"].unflatten(1, (4, 16)), stride)
    k = c["x"].unflatten(1, (4, 16))
    pos, freq, ones = torch.arange(T, dtype=torch.int32, device="cuda"), torch.rand(8, device="cuda"), torch.ones(16, device="cuda")
    a, _ = mm.qk_norm(q, k, ones, ones, pos, freq)
    assert torch.equal(a, mm.qk_norm(k, k, ones, ones, pos, freq)[0])
    mm.qk_norm(q, k, ones, ones, pos, freq, q_out=q)
    assert torch.equal(q, a), "in place, rows far apart"


def many(lens, d):
    """The gated recurrence and the convolution over many sequences, in 64 bits on the GPU, all sequences side by side."""
    c = cuda(ref.gated_inputs(6, lens, d, "f32"))
    S, n = len(lens), max(lens)
    at = torch.zeros(S, n, dtype=torch.long)
    there = torch.zeros(S, n, dtype=torch.bool)
    for s, lo, hi in ref.ranges(lens):
        at[s, :hi - lo] = torch.arange(lo, hi)
        there[s, :hi - lo] = True
    at, there = at.cuda(), there.cuda()
    x, r, g, z = (c[k].double()[at] for k in ("x", "r", "g", "z"))
    a, m, u = ref._gates(x, r, g, c["lam"].double())
    h, mag = c["state"].double(), c["state"].double().abs()
    ys, ms = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(n):
        on = there[:, t, None]
        h = torch.where(on, a[:, t] * h + m[:, t] * u[:, t], h)
        mag = torch.where(on, a[:, t] * mag + (m[:, t] * u[:, t]).abs(), mag)
        ys[:, t], ms[:, t] = h, mag
    o = ref.act(z, "silu")
    y, last = mm.gated_prefill(*[c[k] for k in ("x", "r", "g", "z", "lam", "cu", "state")])
    ref.check(y, (ys * o)[there].cpu(), (ms * o.abs() * (1 + z.abs()))[there].cpu(), n, "y")
    ref.check(last, h.cpu(), mag.cpu(), n, "state")
    w, b, st = torch.randn(d, 4, device="cuda"), torch.randn(d, device="cuda"), torch.randn(S, d, 3, device="cuda")
    X = torch.cat([st.double().transpose(1, 2), x], 1)
    taps = [X[:, k:k + n] * w[:, k].double() for k in range(4)]
    y, last = mm.conv_prefill(c["x"], w, b, c["cu"], st, silu=False)
    ref.check(y, (sum(taps) + b)[there].cpu(), (sum(t.abs() for t in taps) + b.abs())[there].cpu(), 4, "conv")
    ends = torch.tensor(lens, device="cuda")[:, None] + torch.arange(3, device="cuda")
    assert torch.equal(last.double(), X.gather(1, ends[..., None].expand(-1, -1, d)).transpose(1, 2))


def test_many_short_sequences():
    g = torch.Generator().manual_seed(7)
    many([int(v) for v in torch.randint(0, 41, (3000,), generator=g)], 68)


def test_a_long_sequence_among_short_ones():
    many([3, 20000, 0, 1, 65, 64, 128], 36)


def test_long_sequences_repeat_bit_for_bit():
    f, b = gated_calls([30000, 9000], 700, "bf16")
    for call in (f, b):
        first = [t.clone() for t in call()]
        for _ in range(3):
            for a, t in zip(call(), first):
                assert torch.equal(a, t)


def test_checkpoints_of_states_in_place():
    """Sequences that start at a checkpoint, in the middle of a tile or at its start, and end many tiles later or in the next one:
    the checkpoints hold their initial states, which the same call writes over."""
    lens = [64, 128, 64, 2000, 48, 128, 0, 64, 192, 5000, 120, 65, 63, 128]
    c = cuda(ref.gated_inputs(11, lens, 520, "bf16"))
    ins = [c[k] for k in ("x", "r", "g", "z", "lam", "cu")]
    y, last, ckpt = mm.gated_prefill_train(*ins, c["state"])
    starts = c["cu"][:-1].long().tolist()
    for s, t in enumerate(starts):
        if t % mm.layer.GATED_BLOCK == 0 and lens[s] > 0:
            assert torch.equal(ckpt[t // mm.layer.GATED_BLOCK], c["state"][s])
    for _ in range(5):
        st = c["state"].clone()
        got = mm.gated_prefill_train(*ins, st, st)
        assert torch.equal(got[0], y) and torch.equal(st, last) and torch.equal(got[2], ckpt)


def test_more_tokens_than_a_launch_has_threads_for():
    """2^28 + 600 tokens of one head of eight columns, in place: 256 threads to 16 tokens, and at most 2^32 - 1 threads to a launch."""
    T, n = 2 ** 28 + 600, 1000
    g = torch.Generator().manual_seed(5)
    rows = torch.randn(2, n, 1, 8, generator=g, dtype=torch.float32).bfloat16().cuda()
    wq, wk = (torch.rand(8, generator=g).add(0.5).cuda() for _ in range(2))
    q, k = (torch.zeros(T, 1, 8, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    want = mm.qk_norm(rows[0], rows[1], wq, wk)
    for t0 in (0, T // 2, 2 ** 28 - n, 2 ** 28 - 16 - n // 2, T - n):
        q[t0:t0 + n], k[t0:t0 + n] = rows[0], rows[1]
        mm.qk_norm(q, k, wq, wk, q_out=q, k_out=k)
        assert torch.equal(q[t0:t0 + n], want[0]) and torch.equal(k[t0:t0 + n], want[1])


def scan(a, b, h):
    """h_t = a_t h_{t-1} + b_t over the rows of a, b [T, d] from h [d]: blocks of rows side by side, then from block to block."""
    T, n = len(a), 512
    pad = -T % n
    a = torch.cat([a, a.new_ones(pad, a.shape[1])]).unflatten(0, (-1, n))
    b = torch.cat([b, b.new_zeros(pad, b.shape[1])]).unflatten(0, (-1, n))
    A, H = torch.ones_like(a), torch.zeros_like(b)
    A[:, 0], H[:, 0] = a[:, 0], b[:, 0]
    for t in range(1, n):
        A[:, t], H[:, t] = A[:, t - 1] * a[:, t], a[:, t] * H[:, t - 1] + b[:, t]
    for k in range(len(H)):
        H[k] += A[k] * h
        h = H[k, -1]
    return H.flatten(0, 1)[:T]


@pytest.mark.parametrize("lens", [[150000], [90000, 60011]], ids=str)
def test_long_chains(lens):
    """Chains of more than a thousand tiles, with decays that carry a state over several thousand tokens."""
    d = 40
    c = cuda(ref.gated_inputs(9, lens, d, "f32"))
    far = 1.0 - 10.0 ** -torch.linspace(3, 4.5, d, device="cuda", dtype=torch.float64)
    c["lam"] = torch.log(torch.expm1(-torch.log(far) / 8)).float()
    ins = [c[k] for k in ("x", "r", "g", "z", "lam", "cu", "state")]
    y, last, ckpt = mm.gated_prefill_train(*ins)
    got = mm.gated_backward(*ins, c["dy"], c["dstate"], ckpt)
    again = mm.gated_backward(*ins, c["dy"], c["dstate"])
    for s, lo, hi in ref.ranges(lens):
        x, r, g, z, dy = (c[k][lo:hi].double() for k in ("x", "r", "g", "z", "dy"))
        a, m, u = ref._gates(x, r, g, c["lam"].double())
        o, n = ref.act(z, "silu"), hi - lo
        h, mag = scan(a, m * u, c["state"][s].double()), scan(a, (m * u).abs(), c["state"][s].double().abs())
        ref.check(y[lo:hi], (h * o).cpu(), (mag * o.abs() * (1 + z.abs())).cpu(), n, "y")
        ref.check(last[s], h[-1].cpu(), mag[-1].cpu(), n, "state")
        # R_t = a_t G_t, from the last token to the first: R_t = a_t R_{t+1} + a_t dy act
        back, ask = a.flip(0), (dy * o).flip(0)
        R = [scan(back, back * v, w) for v, w in ((ask, c["dstate"][s].double()),
                                                  ((dy * o).abs().mul(1 + z.abs()).flip(0), c["dstate"][s].double().abs()))]
        G, Gm = ((v / back).flip(0) for v in R)
        iota = torch.sigmoid(g)
        for grads in (got, again):
            ref.check(grads["dx"][lo:hi], (G * m * iota).cpu(), (Gm * m * iota).cpu(), n, "dx")
            ref.check(grads["dstate_in"][s], R[0][-1].cpu(), R[1][-1].cpu(), n, "dstate_in")
