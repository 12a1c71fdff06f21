"""The causal convolution, the gated recurrence and the norms of queries and keys in 64 bits, from their definitions, with
the bounds their results are held to.

Bounds.  Every output is a sum of products; `mag` is the same sum over the products' magnitudes, factors that are
differences taken as sums.  An implementation whose products each carry a relative error e is off by at most e mag.
  * float32 arithmetic: e = 2^-23 (24 + 4 sqrt(n)), n the products that are summed or the steps a state runs through: a
    factor of a product is a sigmoid, an exponential or a root with an argument and a result a few units off (24 in all),
    and a rounding per step or summand adds up as a random walk.  A decay's relative error is its exponent's absolute
    one: along a run whose decays multiply to e^-X it is X times the exponent's relative error, at most e^-1 of it
    after the decay itself.
  * each output is rounded once: 2^-8 (bfloat16) or 2^-24 of it.
  * the angle of a rotation: 2^-24 of half a turn after its whole turns are dropped, then the sine's own two units: 2^-21 in
    all of the pair's magnitudes, inside the 24.
"""
from __future__ import annotations

import math

import torch

DT = dict(bf16=torch.bfloat16, f32=torch.float32)
EPS = 1e-5
NAN = float("nan")


def check(got, want, mag, n, what, finite=True):
    g = got.detach().cpu().double()
    assert g.shape == want.shape, f"{what}: shape {tuple(g.shape)}, expected {tuple(want.shape)}"
    if finite:
        assert torch.isfinite(g).all(), f"{what}: not finite"
    if g.numel() == 0:
        return
    half = 2.0 ** -8 if got.dtype == torch.bfloat16 else 2.0 ** -24
    e = 2.0 ** -23 * (24 + 4 * math.sqrt(max(n, 1)))
    worst = float(((g - want).abs() / (half * want.abs() + e * mag + 1e-30)).max())
    assert worst <= 1.0, f"{what}: {worst:.3g} times the bound"


def cu_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)


def gen(seed):
    g = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g)


def ranges(lens):
    at = 0
    for s, n in enumerate(lens):
        yield s, at, at + n
        at += n


# ----------------------------------------------------------------------------------------- convolution
def conv_inputs(seed, lens, d, W, io, bias=True, state=True):
    """CPU tensors; x is a column range of a wider one."""
    r, T, S = gen(seed), sum(lens), len(lens)
    return dict(lens=lens, W=W, cu=cu_of(lens), x=r(T, d + 3).to(DT[io])[:, 3:], weight=r(d, W) * 0.6,
                bias=r(d) if bias else None, state=r(S, d, W - 1) if state else None, dy=r(T, d).to(DT[io]),
                dstate=r(S, d, W - 1))


def conv(c, silu, leaves=None):
    """(y, state_out, mag of y)"""
    x, w, b, state = leaves or [t.double() if t is not None else None for t in (c["x"], c["weight"], c["bias"], c["state"])]
    W, d = c["W"], x.shape[1]
    ys, mags, last = [], [], []
    for s, lo, hi in ranges(c["lens"]):
        X = torch.cat([state[s].T if state is not None else x.new_zeros(W - 1, d), x[lo:hi]])
        taps = [X[k:k + hi - lo] * w[:, k] for k in range(W)]
        u = sum(taps) + (b if b is not None else 0)
        mag = sum(t.abs() for t in taps) + (b.abs() if b is not None else 0)
        y = u * torch.sigmoid(u) if silu else u
        ys.append(y)
        mags.append((1.1 * mag + (u * y).abs()) if silu else mag)  # the slope is at most 1.1; the exponential's argument is u
        last.append(X[hi - lo:].T)
    return torch.cat(ys), torch.stack(last), torch.cat(mags).detach()


def conv_backward(c, silu, dstate=True):
    """{name: (gradient, magnitude)}: the adjoint written out, and with every product's magnitude."""
    x, w, dy = c["x"].double(), c["weight"].double(), c["dy"].double()
    W, d, S = c["W"], x.shape[1], len(c["lens"])
    b = c["bias"].double() if c["bias"] is not None else torch.zeros(d, dtype=torch.float64)
    state = c["state"].double() if c["state"] is not None else torch.zeros(S, d, W - 1, dtype=torch.float64)
    out = {}
    for part in (0, 1):
        mag = (lambda t: t.abs()) if part else (lambda t: t)
        dx, ds = torch.zeros_like(x), torch.zeros(S, d, W - 1, dtype=torch.float64)
        dw, db = torch.zeros_like(w), torch.zeros(d, dtype=torch.float64)
        for s, lo, hi in ranges(c["lens"]):
            n = hi - lo
            X = torch.cat([state[s].T, x[lo:hi]])
            u = sum(X[k:k + n] * w[:, k] for k in range(W)) + b
            um = sum((X[k:k + n] * w[:, k]).abs() for k in range(W)) + b.abs()
            sg = torch.sigmoid(u)
            slope = (sg + mag(u) * sg * (1 - sg)) if silu else torch.ones_like(u)
            g = mag(dy[lo:hi]) * (slope + (um + 1 if part and silu else 0))  # the slope changes by at most u's error
            dX = torch.zeros(n + W - 1, d, dtype=torch.float64)
            for k in range(W):
                dX[k:k + n] += g * mag(w[:, k])
                dw[:, k] += (g * mag(X[k:k + n])).sum(0)
            db += g.sum(0)
            if dstate:
                dX[n:] += mag(c["dstate"][s].double().T)
            ds[s], dx[lo:hi] = dX[:W - 1].T, dX[W - 1:]
        for k, v in dict(dx=dx, dweight=dw, dbias=db, dstate_in=ds).items():
            out.setdefault(k, []).append(v)
    if c["bias"] is None:
        del out["dbias"]
    return out


# ------------------------------------------------------------------------------------ gated recurrence
def gated_inputs(seed, lens, d, io, lam=True, g=True, z=True, state=True, spread=1.0):
    """CPU tensors; x, r, g, z are column ranges of one."""
    r, T, S = gen(seed), sum(lens), len(lens)
    p = r(T, 4 * d + 5)
    p[:, d:2 * d] *= spread
    if not lam:
        p[:, d:2 * d] += 2.0
    p = p.to(DT[io])
    far = 0.9 + 0.0999 * torch.sigmoid(r(d))
    return dict(lens=lens, cu=cu_of(lens), x=p[:, :d], r=p[:, d:2 * d], g=p[:, 2 * d:3 * d] if g else None,
                z=p[:, 3 * d:4 * d] if z else None, lam=torch.log(torch.expm1(-torch.log(far) / 8)) if lam else None,
                state=r(S, d) if state else None, dy=r(T, d).to(DT[io]), dstate=r(S, d))


def act(z, kind):
    k, s = (z, 1.0) if kind == "silu" else (z + 0.044715 * z ** 3, 2 * math.sqrt(2 / math.pi))
    return z * torch.sigmoid(s * k)


def _gates(x, r, g, lam, c=8.0):
    rho = torch.sigmoid(r)
    if lam is None:
        a, m = rho, torch.sigmoid(-r)
    else:
        L = -c * torch.logaddexp(lam, torch.zeros_like(lam)) * rho
        a, m = torch.exp(L), torch.sqrt(-torch.expm1(2 * L))
    return a, m, x * (torch.sigmoid(g) if g is not None else 1.0)


def _run(lens, a, b, state):
    """The states after each token, before each, and the final ones."""
    T, d = a.shape
    after, before, last = [], [], []
    for s, lo, hi in ranges(lens):
        h = state[s]
        for t in range(lo, hi):
            before.append(h)
            h = a[t] * h + b[t]
            after.append(h)
        last.append(h)
    stack = lambda v: torch.stack(v) if v else a.new_zeros(0, d)  # noqa: E731
    return stack(after), stack(before), stack(last)


def _gated_leaves(c):
    dbl = lambda t: t.double() if t is not None else None  # noqa: E731
    st = dbl(c["state"]) if c["state"] is not None else torch.zeros(len(c["lens"]), c["x"].shape[1], dtype=torch.float64)
    return [dbl(c[k]) for k in ("x", "r", "g", "z", "lam")] + [st]


def gated(c, kind="silu", leaves=None):
    """(y, state_out, mag of y, mag of state_out, (the states before each token, their mag))"""
    x, r, g, z, lam, st = leaves or _gated_leaves(c)
    a, m, u = _gates(x, r, g, lam)
    h, before, last = _run(c["lens"], a, m * u, st)
    hm, bm, lm = _run(c["lens"], a.detach(), (m * u).detach().abs(), st.detach().abs())
    if z is None:
        return h, last, hm, lm, (before, bm)
    o = act(z, kind)
    return h * o, last, hm * o.detach().abs() * (1 + z.detach().abs()), lm, (before, bm)


def gated_backward(c, kind="silu", dstate=True, cst=8.0):
    """{name: (gradient, magnitude)}"""
    x, r, g, z, lam, st = _gated_leaves(c)
    rho = torch.sigmoid(r)
    iota = torch.sigmoid(g) if g is not None else torch.ones_like(x)
    a, m, u = _gates(x, r, g, lam)
    dy, lens = c["dy"].double(), c["lens"]
    ds = c["dstate"].double() if dstate else torch.zeros_like(st)
    if z is not None:
        zz = z.clone().requires_grad_(True)
        o = act(zz, kind)
        slope = torch.autograd.grad(o.sum(), zz)[0]
        o = o.detach()
        steep = (1 + z.abs()) * (1 + z.abs())  # what the slope's two terms add up to, and their arguments
    out = {}
    for part in (0, 1):
        mag = (lambda t: t.abs()) if part else (lambda t: t)
        after, before, _ = _run(lens, a, mag(m * u), mag(st))
        dh = mag(dy * o if z is not None else dy) * (1 + z.abs() if part and z is not None else 1)
        G, first = torch.zeros_like(dh), []
        for s, lo, hi in ranges(lens):
            v = mag(ds[s])
            for t in reversed(range(lo, hi)):
                v = v + dh[t]
                G[t] = v
                v = a[t] * v
            first.append(v)
        res = dict(dx=G * m * iota, dstate_in=torch.stack(first))
        if g is not None:
            res["dg"] = G * m * mag(u) * (1 - iota)
        if z is not None:
            res["dz"] = mag(dy) * after * (steep if part else slope)
        if lam is None:
            res["dr"] = G * (before - u if not part else before + u.abs()) * rho * (1 - rho)
        else:
            sp = torch.logaddexp(lam, torch.zeros_like(lam))
            L = -cst * sp * rho
            q = torch.where(L < 0, L / torch.where(m > 0, m, 1.0), 0.0)
            e = G * (a * before * L - u * a * a * q) if not part else G * (a * before * L.abs() + u.abs() * a * a * q.abs())
            res["dr"] = e * (1 - rho)
            res["dlam"] = e.sum(0) * torch.sigmoid(lam) / sp
        for k, v in res.items():
            out.setdefault(k, []).append(v)
    return out


# ------------------------------------------------------------------------------- queries and keys' norms
def qk_inputs(seed, T, Hq, Hk, D, R, io, far=1 << 20):
    r = gen(seed)
    p = r(T, (Hq + Hk) * D + 3).to(DT[io])
    pos = (torch.rand(T, generator=torch.Generator().manual_seed(seed)) * far).to(torch.int32)
    return dict(q=p[:, :Hq * D].unflatten(1, (Hq, D)), k=p[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)), wq=1 + 0.1 * r(D),
                wk=1 + 0.1 * r(D), pos=pos if R else None,
                freq=10000.0 ** (-torch.arange(R // 2) * 2.0 / R) if R else None, R=R,
                dq=r(T, Hq, D).to(DT[io]), dk=r(T, Hk, D).to(DT[io]))


def turned(v, c, inter, sign=1.0, mag=False):
    R = c["R"]
    if not R:
        return v
    f = c["pos"].double()[:, None] * c["freq"].double()
    co, si = torch.cos(f)[:, None], sign * torch.sin(f)[:, None]
    i = torch.arange(R // 2)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + R // 2)
    out = v.clone()
    if mag:  # the angle's error moves either by the other: both count whole
        out[..., a] = out[..., b] = v[..., a] + v[..., b]
        return out
    out[..., a] = v[..., a] * co - v[..., b] * si
    out[..., b] = v[..., b] * co + v[..., a] * si
    return out


def qk(c, inter, eps=EPS):
    """[(out, mag)] of queries and keys"""
    res = []
    for v, w in ((c["q"].double(), c["wq"].double()), (c["k"].double(), c["wk"].double())):
        u = v / torch.sqrt((v ** 2).mean(-1, keepdim=True) + eps) * w
        res.append((turned(u, c, inter), turned(u.abs(), c, inter, mag=True)))
    return res


def qk_backward(c, inter, eps=EPS):
    """{name: (gradient, magnitude)}"""
    out = {}
    for name, v, w, do in (("q", c["q"], c["wq"], c["dq"]), ("k", c["k"], c["wk"], c["dk"])):
        v, w, do = v.double(), w.double(), do.double()
        k = 1 / torch.sqrt((v ** 2).mean(-1, keepdim=True) + eps)
        n = v * k
        g, gm = turned(do, c, inter, -1.0), turned(do.abs(), c, inter, mag=True)
        dn, dm = g * w, gm * w.abs()
        out["d" + name] = (k * (dn - n * (dn * n).mean(-1, keepdim=True)), k * (dm + n.abs() * (dm * n.abs()).mean(-1, keepdim=True)))
        out["dw" + name] = ((g * n).sum((0, 1)), (gm * n.abs()).sum((0, 1)))
    return out
