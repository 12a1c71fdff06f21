"""The head scan and the norms in 64 bits, token by token, with the bounds their float32 and bfloat16
results are held to.

Bounds.  Every output is a sum of products.  `mag` is the same sum over the products' magnitudes (the
recurrence run on absolute values), so an implementation whose products each carry a relative error e
is off by at most e mag.
  * float32 results: e = 2^-23 (16 + 4 sqrt(T)): a few roundings per product (the decays' exponents among
    them), and a rounding per step that adds up as a random walk along T steps.
  * bfloat16 results (8 significant bits: rounding to nearest is off by at most 2^-8): the final rounding,
    2^-8 |r|, and products of which one factor may have been rounded to bfloat16: e = 2^-8.
  * sums over tokens of bfloat16 paths (dA_log, ddt_bias, dD): float32 results, the float32 bound.
"""
from __future__ import annotations

import math

import torch

F32_EPS = 2.0 ** -23


def heads_inputs(seed, lens, H, P, G, N, io, dt=True, D=True, state=True):
    """Token tensors as column ranges of one projection output (strided rows), on the CPU."""
    g = torch.Generator().manual_seed(seed)
    T, S, d = sum(lens), len(lens), H * P
    proj = torch.randn(T, 2 * d + 2 * G * N + H, generator=g)
    proj[:, 2 * d:2 * d + 2 * G * N] *= N ** -0.25
    proj = proj.to(torch.bfloat16 if io == "bf16" else torch.float32)
    c = dict(lens=lens, H=H, P=P, G=G, N=N, io=io, proj=proj,
             cu=torch.tensor([sum(lens[:i]) for i in range(S + 1)], dtype=torch.int32),
             A_log=torch.log(1 + 15 * torch.rand(H, generator=g)),
             D=1 + 0.1 * torch.randn(H, generator=g) if D else None,
             dt_bias=-4 + 2 * torch.rand(H, generator=g) if dt else None,
             state=0.5 * torch.randn(S, H, P, N, generator=g) if state else None,
             dy=torch.randn(T, H, P, generator=g).to(proj.dtype),
             dstate=0.5 * torch.randn(S, H, P, N, generator=g))
    return split(c, dt)


def split(c, dt=True):
    """The token tensors as views of c["proj"] (again, after moving it)."""
    H, P, G, N, p = c["H"], c["P"], c["G"], c["N"], c["proj"]
    d, w = H * P, G * N
    c["x"] = p[:, d:2 * d].unflatten(1, (H, P))
    c["B"] = p[:, 2 * d:2 * d + w].unflatten(1, (G, N))
    c["C"] = p[:, 2 * d + w:2 * d + 2 * w].unflatten(1, (G, N))
    c["dt"] = p[:, 2 * d + 2 * w:] if dt else None
    return c


def _tokens(c):
    x, B, C = c["x"].double(), c["B"].double(), c["C"].double()
    hg = c["H"] // c["G"]
    B, C = B.repeat_interleave(hg, 1), C.repeat_interleave(hg, 1)
    A = -torch.exp(c["A_log"].double())
    if c["dt"] is None:
        v, delta = None, torch.ones(x.shape[:2], dtype=torch.float64)
    else:
        v = c["dt"].double() + c["dt_bias"].double()
        delta = torch.logaddexp(v, torch.zeros_like(v))
    D = c["D"].double() if c["D"] is not None else torch.zeros(c["H"], dtype=torch.float64)
    return x, B, C, A, v, delta, D


def _state(c, key="state"):
    s = c[key]
    return s.double() if s is not None else torch.zeros(len(c["lens"]), c["H"], c["P"], c["N"], dtype=torch.float64)


def forward(c):
    """(y, state_out, mag of y, mag of state_out)"""
    x, B, C, A, _, delta, D = _tokens(c)
    h = _state(c)
    y, ya = torch.empty_like(x), torch.empty_like(x)
    hs, ms = [], []
    at = 0
    for s, n in enumerate(c["lens"]):
        cur, mag = h[s], h[s].abs()
        for t in range(at, at + n):
            a = torch.exp(A * delta[t])[:, None, None]
            new = (delta[t][:, None] * x[t])[:, :, None] * B[t][:, None, :]
            cur, mag = a * cur + new, a * mag + new.abs()
            y[t] = (cur @ C[t][:, :, None])[..., 0] + D[:, None] * x[t]
            ya[t] = (mag @ C[t].abs()[:, :, None])[..., 0] + (D[:, None] * x[t]).abs()
        hs.append(cur)
        ms.append(mag)
        at += n
    return y, torch.stack(hs), ya, torch.stack(ms)


def _adjoint(x, B, C, A, delta, D, h0, dy, dh, lens, sign):
    """The gradients by the recurrence's adjoint; sign=1: the values, sign=0: their magnitudes."""
    f = (lambda v: v) if sign else torch.abs
    x, B, C, D, h0, dy, dh = (f(v) for v in (x, B, C, D, h0, dy, dh))
    Am = A if sign else A.abs()
    dx, dB, dC = torch.empty_like(x), torch.empty_like(B), torch.empty_like(C)
    r, dl, q, p = (torch.empty_like(delta) for _ in range(4))
    dh0 = []
    at = 0
    for s, n in enumerate(lens):
        states = [h0[s]]
        for t in range(at, at + n):
            states.append(torch.exp(A * delta[t])[:, None, None] * states[-1]
                          + (delta[t][:, None] * x[t])[:, :, None] * B[t][:, None, :])
        g = dh[s]
        for t in reversed(range(at, at + n)):
            new, old = states[t - at + 1], states[t - at]
            g = g + dy[t][:, :, None] * C[t][:, None, :]
            dC[t] = (dy[t][:, None, :] @ new)[:, 0]
            gB = (g @ B[t][:, :, None])[..., 0]
            dB[t] = delta[t][:, None] * (x[t][:, None, :] @ g)[:, 0]
            dx[t] = delta[t][:, None] * gB + D[:, None] * dy[t]
            r[t] = (x[t] * gB).sum(1)
            q[t] = (dC[t] * C[t]).sum(1)
            p[t] = delta[t] * r[t]
            g = torch.exp(A * delta[t])[:, None, None] * g
            dl[t] = (g * old).sum((1, 2))
        dh0.append(g)
        at += n
    if not sign:  # inside 64-token blocks dl is a sum of q - p from the block's end: their magnitudes count
        at = 0
        for n in lens:
            for b in range(at // 64, (at + n - 1) // 64 + 1 if n else 0):
                t0, t1 = max(at, 64 * b), min(at + n, 64 * b + 64)
                dl[t0:t1] += (q[t0:t1] + p[t0:t1]).sum(0)
            at += n
    return dx, dB, dC, r + Am * dl, delta * dl * Am, torch.stack(dh0)


def backward(c, dstate=True):
    """{name: (gradient, magnitude)}"""
    x, B, C, A, v, delta, D = _tokens(c)
    dh = c["dstate"].double() if dstate else torch.zeros_like(c["dstate"], dtype=torch.float64)
    dy, h0 = c["dy"].double(), _state(c)
    out = {}
    both = [_adjoint(x, B, C, A, delta, D, h0, dy, dh, c["lens"], sign) for sign in (1, 0)]
    G, hg = c["G"], c["H"] // c["G"]
    share = lambda t: t.unflatten(1, (G, hg)).sum(2)  # noqa: E731
    sig = torch.sigmoid(v) if v is not None else None
    for name, fn in (("dx", lambda t: t[0]), ("dB", lambda t: share(t[1])), ("dC", lambda t: share(t[2])),
                     ("dA_log", lambda t: t[4].sum(0)), ("dstate_in", lambda t: t[5])):
        out[name] = tuple(fn(t) for t in both)
    if sig is not None:
        out["ddt"] = tuple(t[3] * sig for t in both)
        out["ddt_bias"] = tuple((t[3] * sig).sum(0) for t in both)
    if c["D"] is not None:
        out["dD"] = ((x * dy).sum((0, 2)), (x * dy).abs().sum((0, 2)))
    return out


def bound(r, mag, dtype, T):
    if dtype == torch.bfloat16:
        return 2.0 ** -8 * (r.abs() + mag) + 1e-30
    return F32_EPS * (16 + 4 * math.sqrt(max(T, 1))) * mag + 1e-30


def check(got, r, mag, T, what):
    g = got.detach().cpu().double()
    assert g.shape == r.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(r.shape)}"
    assert torch.isfinite(g).all(), f"{what}: not finite"
    if g.numel() == 0:
        return 0.0
    worst = float(((g - r).abs() / bound(r, mag, got.dtype, T)).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"
    return worst


# ------------------------------------------------------------------------------------------ norms
EPS = 1e-5


def _norm(u):
    return u / torch.sqrt((u ** 2).mean(-1, keepdim=True) + EPS)


def gate_norm(y, z, w, groups, gate_first):
    s = z * torch.sigmoid(z)
    shape = (y.shape[0], groups, -1) if y.shape[0] else (0, groups, y.shape[1] // groups)
    out = _norm((y * s if gate_first else y).reshape(shape)).reshape(y.shape) * w
    return out if gate_first else out * s


def residual_norm(h, r, w, wp, scale, vec):
    p = _norm(h) * wp if wp is not None else h
    new = r + (scale * vec if vec is not None else scale) * p
    return _norm(new) * w, new


def check_rows(got, r, terms, what):
    """One rounding of the result (2^-8 bfloat16, 2^-24 float32), and float32 arithmetic: 2^-23 times the sum of
    the magnitudes of its `terms` (each term's row statistics included), times 16 roundings."""
    g = got.detach().cpu().double()
    assert g.shape == r.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(r.shape)}"
    assert torch.isfinite(g).all(), f"{what}: not finite"
    if g.numel() == 0:
        return
    e = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    worst = float(((g - r).abs() / (e * r.abs() + 16 * F32_EPS * terms + 1e-30)).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"
