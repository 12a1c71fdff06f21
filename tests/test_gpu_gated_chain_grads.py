"""All gradients of the gated recurrence over chains of more than a thousand tiles, in 64 bits on the GPU.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref
from tests.test_gpu_layer_calls import cuda, scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lam", [True, False])
@pytest.mark.parametrize("lens", [[150000], [90000, 60011]], ids=str)
def test_gradients(lens, lam):
    d, T = 40, sum(lens)
    c = cuda(ref.gated_inputs(12, lens, d, "f32", lam))
    if lam:  # decays that carry a state over several thousand tokens
        far = 1.0 - 10.0 ** -torch.linspace(3, 4.5, d, device="cuda", dtype=torch.float64)
        c["lam"] = torch.log(torch.expm1(-torch.log(far) / 8)).float()
    else:
        c["r"] = c["r"] + 6.0
    ins = [c[k] for k in ("x", "r", "g", "z", "lam", "cu", "state")]
    got = mm.gated_backward(*ins, c["dy"], c["dstate"])
    want = {}
    for s, lo, hi in ref.ranges(lens):
        x, r, g, z, dy = (c[k][lo:hi].double() for k in ("x", "r", "g", "z", "dy"))
        L0 = c["lam"].double() if lam else None
        a, m, u = ref._gates(x, r, g, L0)
        rho, iota, state = torch.sigmoid(r), torch.sigmoid(g), c["state"][s].double()
        zz = z.clone().requires_grad_(True)
        o = ref.act(zz, "silu")
        slope, o, steep = torch.autograd.grad(o.sum(), zz)[0], o.detach(), (1 + z.abs()) ** 2
        for part in (0, 1):
            mag = (lambda t: t.abs()) if part else (lambda t: t)
            h = scan(a, mag(m * u), mag(state))
            before = torch.cat([mag(state)[None], h[:-1]])
            ask = mag(dy * o) * (1 + z.abs() if part else 1)
            back = a.flip(0)
            G = (scan(back, back * ask.flip(0), mag(c["dstate"][s].double())) / back).flip(0)  # R_t = a_t G_t
            res = dict(dx=G * m * iota, dg=G * m * mag(u) * (1 - iota), dz=mag(dy) * h * (steep if part else slope))
            if lam:
                sp = torch.logaddexp(L0, torch.zeros_like(L0))
                L = -8.0 * sp * rho
                e = G * (a * before * mag(L) + (1 if part else -1) * mag(u) * a * a * mag(L) / m)
                res["dr"] = e * (1 - rho)
                res["dlam"] = e.sum(0) * torch.sigmoid(L0) / sp
            else:
                res["dr"] = G * (before + (1 if part else -1) * mag(u)) * rho * (1 - rho)
            for k, v in res.items():
                want.setdefault(k, ([], []))[part].append(v)
    for k, (v, mag) in want.items():
        v, mag = (sum(t) if k == "dlam" else torch.cat(t) for t in (v, mag))
        ref.check(got[k], v.cpu(), mag.cpu(), T, k)
