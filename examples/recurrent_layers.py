"""Two recurrent layers as a model would run them, with the convolution ahead of each.

`GatedLayer`, one decay and one state per channel:

    n, res = residual_norm(h, res)               the residual stream takes the last layer's output h
    x, z   = column ranges of n W_in
    u      = conv_prefill(x)
    r, g   = column ranges of u W_gates          the gates come from the convolution's output
    h      = gated_prefill(u, r, g, z) W_out

`RetentionLayer`, one fixed decay per head, its queries and keys normalised and turned by position:

    n, res  = residual_norm(h, res)
    z, xBC  = column ranges of n W_in
    u       = conv_prefill(xBC), SiLU            u = x | B | C
    q, k    = qk_norm(C, B) at the tokens' positions
    h       = gate_norm(heads_prefill(x, k, q), z) W_out

`prefill` takes packed sequences and leaves their states, `step` continues them a token at a time in place (a HIP graph may
hold it), `backward` gives the gradients of a prefill.  The products are the caller's own (torch's here).

    python examples/recurrent_layers.py          three prompts, 32 generated tokens, one training step
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_causal_amd as mm  # noqa: E402

TAPS = 4


def _random(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g)


class GatedLayer:
    """hidden columns in and out, d channels."""

    names = ("norm", "w_in", "conv_w", "conv_b", "w_gates", "lam", "w_out")

    def __init__(self, hidden, d, dtype=torch.bfloat16, device="cuda", seed=0):
        rnd, self.d = _random(seed), d
        far = 0.9 + 0.099 * torch.sigmoid(rnd(d))  # the decay of a fully open gate
        self.norm = (1 + 0.1 * rnd(hidden)).to(device)
        self.w_in = (rnd(hidden, 2 * d) * hidden ** -0.5).to(device, dtype)
        self.conv_w, self.conv_b = (rnd(d, TAPS) * 0.5).to(device), (0.1 * rnd(d)).to(device)
        self.w_gates = (rnd(d, 2 * d) * d ** -0.5).to(device, dtype)
        self.lam = torch.log(torch.expm1(-torch.log(far) / 8)).to(device)
        self.w_out = (rnd(d, hidden) * d ** -0.5).to(device, dtype)

    def state(self, rows, device="cuda"):
        return torch.zeros(rows, self.d, TAPS - 1, device=device), torch.zeros(rows, self.d, device=device)

    def prefill(self, h, residual, cu, state, positions=None):
        """(out, residual, state, what backward needs); positions are not used."""
        d = self.d
        n, res = mm.residual_norm(h, residual, self.norm)
        p = n @ self.w_in
        u, conv = mm.conv_prefill(p[:, :d], self.conv_w, self.conv_b, cu, state[0], silu=False)
        gates = u @ self.w_gates
        y, last, ckpt = mm.gated_prefill_train(u, gates[:, :d], gates[:, d:], p[:, d:], self.lam, cu, state[1], gate="gelu")
        return y @ self.w_out, res, (conv, last), dict(h=h, n=n, res=res, p=p, u=u, gates=gates, y=y, ckpt=ckpt, cu=cu, state=state)

    def step(self, h, residual, state, positions=None):
        """One token for each row; residual and state are updated in place."""
        d, (conv, last) = self.d, state
        n, _ = mm.residual_norm(h, residual, self.norm, residual_out=residual)
        p = n @ self.w_in
        u, _ = mm.conv_decode(p[:, :d], self.conv_w, self.conv_b, conv, state_out=conv, silu=False)
        gates = u @ self.w_gates
        y, _ = mm.gated_decode(u, gates[:, :d], gates[:, d:], p[:, d:], self.lam, last, state_out=last, gate="gelu")
        return y @ self.w_out

    def backward(self, kept, dout, dres, dstate=(None, None)):
        """From the gradients of prefill's out, residual and state those of its inputs and the parameters."""
        d, p, gates = self.d, kept["p"], kept["gates"]
        got = dict(w_out=kept["y"].t() @ dout)
        dp, dgates = torch.empty_like(p), torch.empty_like(gates)
        s = mm.gated_backward(kept["u"], gates[:, :d], gates[:, d:], p[:, d:], self.lam, kept["cu"], kept["state"][1],
                              dout @ self.w_out.t(), dstate[1], ckpt=kept["ckpt"], gate="gelu", dr=dgates[:, :d],
                              dg=dgates[:, d:], dz=dp[:, d:])
        got.update(lam=s["dlam"], w_gates=kept["u"].t() @ dgates)
        du = s["dx"] + dgates @ self.w_gates.t()
        c = mm.conv_backward(p[:, :d], self.conv_w, self.conv_b, kept["cu"], kept["state"][0], du, dstate[0], silu=False, dx=dp[:, :d])
        got.update(conv_w=c["dweight"], conv_b=c["dbias"], state=(c["dstate_in"], s["dstate_in"]), w_in=kept["n"].t() @ dp)
        b = mm.residual_norm_backward(dp @ self.w_in.t(), dres, kept["h"], kept["res"], self.norm)
        got.update(norm=b["dweight"], h=b["dh"], residual=b["dresidual"])
        return got


class RetentionLayer:
    """hidden columns in and out; H heads of P channels, G groups of queries and keys of N columns."""

    names = ("norm", "w_in", "conv_w", "conv_b", "q_norm", "k_norm", "A_log", "gate", "w_out")

    def __init__(self, hidden, H, P, G, N, dtype=torch.bfloat16, device="cuda", seed=0):
        rnd, self.sizes = _random(seed), (H, P, G, N)
        d, w = H * P, H * P + 2 * G * N
        self.norm = (1 + 0.1 * rnd(hidden)).to(device)
        self.w_in = (rnd(hidden, d + w) * hidden ** -0.5).to(device, dtype)
        self.conv_w, self.conv_b = (rnd(w, TAPS) * 0.5).to(device), (0.1 * rnd(w)).to(device)
        self.q_norm, self.k_norm = ((1 + 0.1 * rnd(N)).to(device) * N ** -0.5, (1 + 0.1 * rnd(N)).to(device) * N ** -0.5)
        self.A_log = torch.log(-torch.log(1 - 2.0 ** (-3 - torch.arange(H) * 4.0 / H))).to(device)  # decays 1 - 2^-3 ...
        self.freq = (10000.0 ** (-torch.arange(N // 2) * 2.0 / N)).to(device)
        self.gate = (1 + 0.1 * rnd(d)).to(device)
        self.w_out = (rnd(d, hidden) * d ** -0.5).to(device, dtype)

    def state(self, rows, device="cuda"):
        H, P, G, N = self.sizes
        return torch.zeros(rows, H * P + 2 * G * N, TAPS - 1, device=device), torch.zeros(rows, H, P, N, device=device)

    def _parts(self, u):
        """x, B, C of the convolution's output."""
        H, P, G, N = self.sizes
        x, B, C = u.split([H * P, G * N, G * N], 1)
        return x.unflatten(1, (H, P)), B.unflatten(1, (G, N)), C.unflatten(1, (G, N))

    def prefill(self, h, residual, cu, state, positions):
        d = self.sizes[0] * self.sizes[1]
        n, res = mm.residual_norm(h, residual, self.norm)
        p = n @ self.w_in
        u, conv = mm.conv_prefill(p[:, d:], self.conv_w, self.conv_b, cu, state[0])
        x, B, C = self._parts(u)
        q, k = mm.qk_norm(C, B, self.q_norm, self.k_norm, positions, self.freq)
        y, last = mm.heads_prefill(x, None, k, q, self.A_log, None, None, cu, state[1])
        out = mm.gate_norm(y.flatten(1), p[:, :d], self.gate, groups=self.sizes[2])
        return out @ self.w_out, res, (conv, last), dict(h=h, n=n, res=res, p=p, u=u, q=q, k=k, y=y, out=out, cu=cu, state=state, pos=positions)

    def step(self, h, residual, state, positions):
        d, (conv, last) = self.sizes[0] * self.sizes[1], state
        n, _ = mm.residual_norm(h, residual, self.norm, residual_out=residual)
        p = n @ self.w_in
        u, _ = mm.conv_decode(p[:, d:], self.conv_w, self.conv_b, conv, state_out=conv)
        x, B, C = self._parts(u)
        q, k = mm.qk_norm(C, B, self.q_norm, self.k_norm, positions, self.freq)
        y, _ = mm.heads_decode(x, None, k, q, self.A_log, None, None, last, state_out=last)
        return mm.gate_norm(y.flatten(1), p[:, :d], self.gate, groups=self.sizes[2]) @ self.w_out

    def backward(self, kept, dout, dres, dstate=(None, None)):
        d, p = self.sizes[0] * self.sizes[1], kept["p"]
        x, B, C = self._parts(kept["u"])
        got = dict(w_out=kept["out"].t() @ dout)
        dp, du = torch.empty_like(p), torch.empty_like(kept["u"])
        dx, dB, dC = self._parts(du)
        dy, _, got["gate"] = mm.gate_norm_backward(dout @ self.w_out.t(), kept["y"].flatten(1), p[:, :d], self.gate,
                                                   groups=self.sizes[2], dz=dp[:, :d])
        s = mm.heads_backward(x, None, kept["k"], kept["q"], self.A_log, None, None, kept["cu"], kept["state"][1],
                              dy.view_as(kept["y"]), dstate[1], dx=dx)
        _, _, got["q_norm"], got["k_norm"] = mm.qk_norm_backward(s["dC"], s["dB"], C, B, self.q_norm, self.k_norm, kept["pos"],
                                                                 self.freq, dq=dC, dk=dB)
        c = mm.conv_backward(p[:, d:], self.conv_w, self.conv_b, kept["cu"], kept["state"][0], du, dstate[0], dx=dp[:, d:])
        got.update(A_log=s["dA_log"], conv_w=c["dweight"], conv_b=c["dbias"], state=(c["dstate_in"], s["dstate_in"]),
                   w_in=kept["n"].t() @ dp)
        b = mm.residual_norm_backward(dp @ self.w_in.t(), dres, kept["h"], kept["res"], self.norm)
        got.update(norm=b["dweight"], h=b["dh"], residual=b["dresidual"])
        return got


def main():
    dev, hidden, lens = "cuda", 2048, [700, 1, 323]
    layers = [GatedLayer(hidden, 2048, seed=0), GatedLayer(hidden, 2048, seed=1), RetentionLayer(hidden, 32, 64, 8, 128, seed=2)]
    T, S = sum(lens), len(lens)
    cu = torch.tensor([sum(lens[:i]) for i in range(S + 1)], dtype=torch.int32, device=dev)
    positions = torch.cat([torch.arange(n) for n in lens]).to(dev, torch.int32)
    h = _random(5)(T, hidden).to(dev, torch.bfloat16)
    r = torch.zeros(T, hidden, device=dev)  # a float32 residual stream
    fresh = [b.state(S) for b in layers]

    def forward():
        x, res, states, kept = h, r, [], []
        for b, s in zip(layers, fresh):
            x, res, s, k = b.prefill(x, res, cu, s, positions)
            states.append(s)
            kept.append(k)
        return x, states, kept

    def timed(f, reps=5):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            got = f()
        torch.cuda.synchronize()
        return got, (time.perf_counter() - t) / reps * 1e6

    (out, states, kept), us = timed(forward)
    print(f"prefill: {T} tokens in {S} sequences, {len(layers)} layers: {us:.0f} us")
    last, at = out[cu[1:].long() - 1].clone(), cu[1:] - cu[:-1]

    def token():
        x, res = last, torch.zeros(S, hidden, device=dev)
        for b, s in zip(layers, states):
            x = b.step(x, res, s, at)
        last.copy_(x)
        at.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token()
    _, us = timed(graph.replay, 31)
    print(f"decode: {S} rows, {len(layers)} layers, captured: {us:.0f} us a token; finite: {bool(last.isfinite().all())}")

    def training():
        dx, dres = torch.ones_like(out), None
        for b, k in zip(reversed(layers), reversed(kept)):
            grads = b.backward(k, dx, dres)
            dx, dres = grads["h"], grads["residual"]
        return dx

    dx, us = timed(training)
    print(f"backward: {us:.0f} us; finite: {bool(dx.isfinite().all())}")


if __name__ == "__main__":
    main()
