"""A layer made of the head scan and the norms around it, as a model would run it.

    n, r  = residual_norm(h, r)                 the residual stream r takes the last layer's output h
    z, x, B, C, dt = column ranges of n W_in    one product; the scan reads its ranges in place
    y, s  = heads_prefill(x, dt, B, C, ..., s)  or heads_decode, one token for each row
    h     = gate_norm(y, z) W_out

`prefill` takes packed sequences and leaves their states, `step` continues them a token at a time with the
states updated in place (it allocates from the caching allocator only, so a HIP graph may hold it), and
`backward` gives the gradients of a prefill.  The products are the caller's own (torch's here).

    python examples/heads_block.py              three prompts, 32 generated tokens, one training step
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import selective_state_space_causal_amd as mm  # noqa: E402


class HeadsBlock:
    """hidden columns in and out; H heads of P channels, G groups of N state entries."""

    def __init__(self, hidden, H, P, G, N, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)
        d, self.sizes = H * P, (H, P, G, N)
        self.widths = [d, d, G * N, G * N, H]  # z, x, B, C, dt
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.w_in = (rnd(hidden, sum(self.widths)) * hidden ** -0.5).to(device, dtype)
        self.w_out = (rnd(d, hidden) * d ** -0.5).to(device, dtype)
        f32 = dict(
            norm=1 + 0.1 * rnd(hidden),
            gate=1 + 0.1 * rnd(d),
            A_log=torch.log(1 + 15 * torch.rand(H, generator=g)),
            D=torch.ones(H),
            dt_bias=-4 + 2 * torch.rand(H, generator=g),
        )
        self.norm, self.gate, self.A_log, self.D, self.dt_bias = (t.to(device) for t in f32.values())

    def _ranges(self, u):
        """z, x, B, C and dt as views of the product's columns."""
        H, P, G, N = self.sizes
        z, x, B, C, dt = u.split(self.widths, 1)
        return z, x.unflatten(1, (H, P)), B.unflatten(1, (G, N)), C.unflatten(1, (G, N)), dt

    def _finish(self, y, z):
        g = mm.gate_norm(y.flatten(1), z, self.gate, groups=self.sizes[2])
        return g, g @ self.w_out

    def prefill(self, h, residual, cu, state=None):
        """h [T, hidden], residual [T, hidden] (or None), cu [S+1], state [S, H, P, N] (None: zeros).
        Returns (h, residual, state) and what `backward` needs."""
        n, r = mm.residual_norm(h, residual, self.norm)
        u = n @ self.w_in
        z, x, B, C, dt = self._ranges(u)
        y, out_state = mm.heads_prefill(x, dt, B, C, self.A_log, self.D, self.dt_bias, cu, state)
        g, out = self._finish(y, z)
        return out, r, out_state, dict(h=h, n=n, r=r, u=u, y=y, g=g, cu=cu, state=state)

    def step(self, h, residual, state):
        """One token for each row: h, residual [Bs, hidden]; residual and state are updated in place."""
        n, r = mm.residual_norm(h, residual, self.norm, residual_out=residual)
        z, x, B, C, dt = self._ranges(n @ self.w_in)
        y, _ = mm.heads_decode(x, dt, B, C, self.A_log, self.D, self.dt_bias, state, state_out=state)
        return self._finish(y, z)[1]

    def backward(self, kept, dout, dr, dstate=None):
        """From the gradients of prefill's h, residual and state (dr and dstate may be None) those of its
        inputs and of the parameters."""
        z, x, B, C, dt = self._ranges(kept["u"])
        du = torch.empty_like(kept["u"])
        dz, dx, dB, dC, ddt = self._ranges(du)  # the operators write the product's gradient in place
        got = dict(w_out=kept["g"].t() @ dout)
        dy, _, got["gate"] = mm.gate_norm_backward(
            dout @ self.w_out.t(), kept["y"].flatten(1), z, self.gate, groups=self.sizes[2], dz=dz)
        s = mm.heads_backward(
            x, dt, B, C, self.A_log, self.D, self.dt_bias, kept["cu"], kept["state"], dy.view_as(kept["y"]), dstate,
            dx=dx, ddt=ddt, dB=dB, dC=dC, need_dstate=kept["state"] is not None)
        got.update(A_log=s["dA_log"], D=s["dD"], dt_bias=s["ddt_bias"], state=s["dstate_in"])
        got["w_in"] = kept["n"].t() @ du
        b = mm.residual_norm_backward(du @ self.w_in.t(), dr, kept["h"], kept["r"], self.norm)
        got.update(norm=b["dweight"], h=b["dh"], residual=b["dresidual"])
        return got


def main():
    dev, hidden, layers, lens = "cuda", 2048, 4, [700, 1, 323]
    H, P, G, N = 64, 64, 8, 128
    blocks = [HeadsBlock(hidden, H, P, G, N, seed=i) for i in range(layers)]
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=dev)
    g = torch.Generator().manual_seed(1)
    h = torch.randn(sum(lens), hidden, generator=g).to(dev, torch.bfloat16)
    r = torch.zeros(sum(lens), hidden, device=dev)  # a float32 residual stream

    def forward():
        x, res, states, kept = h, r, [], []
        for b in blocks:
            x, res, s, k = b.prefill(x, res, cu)
            states.append(s)
            kept.append(k)
        return x, res, states, kept

    def timed(f, reps=5):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(reps):
            got = f()
        torch.cuda.synchronize()
        return got, (time.perf_counter() - t) / reps * 1e6

    (out, _, states, kept), us = timed(forward)
    print(f"prefill: {sum(lens)} tokens in {len(lens)} sequences, {layers} layers: {us:.0f} us")

    last = out[cu[1:].long() - 1].clone()  # "the next token" of each sequence: its last output

    def token():
        x, res = last, torch.zeros(len(lens), hidden, device=dev)
        for b, s in zip(blocks, states):
            x = b.step(x, res, s)
        last.copy_(x)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        token()
    _, us = timed(graph.replay, 31)
    print(f"decode: {len(lens)} rows, {layers} layers, captured: {us:.0f} us a token; finite: {bool(last.isfinite().all())}")

    def training():
        dx, dres = torch.ones_like(out), None
        for b, k in zip(reversed(blocks), reversed(kept)):
            grads = b.backward(k, dx, dres)
            dx, dres = grads["h"], grads["residual"]
        return dx

    dx, us = timed(training)
    print(f"backward: {us:.0f} us; finite: {bool(dx.isfinite().all())}")


if __name__ == "__main__":
    main()
