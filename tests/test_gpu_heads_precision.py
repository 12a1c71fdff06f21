"""The parameters' gradients of the head scan are float32 results: they are held to the error that the same
recurrence and its adjoint have in float32 arithmetic throughout.  The kernels make no more roundings per term than that, so
over several inputs their errors are of its size; three times allows for chance.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

from tests import heads_ref as ref
from tests.gpu_util import log
from tests.test_gpu_heads import run_backward

pytestmark = pytest.mark.gpu

NAMES = dict(A_log="dA_log", dt_bias="ddt_bias", D="dD", state="dstate_in")


def gradients(c, dtype):
    """Through torch's differentiation of the recurrence, token by token, in one type."""
    H, G = c["H"], c["G"]
    t = {k: c[k].to(dtype) for k in ("x", "dt", "B", "C", "dy", "dstate")}
    p = {k: c[k].to(dtype).clone().requires_grad_() for k in NAMES}
    B, C = (t[k].repeat_interleave(H // G, 1) for k in "BC")
    delta = torch.nn.functional.softplus(t["dt"] + p["dt_bias"], threshold=700)
    a = torch.exp(-torch.exp(p["A_log"]) * delta)
    loss, at = 0, 0
    for s, n in enumerate(c["lens"]):
        h = p["state"][s]
        for i in range(at, at + n):
            h = a[i][:, None, None] * h + (delta[i][:, None] * t["x"][i])[:, :, None] * B[i][:, None, :]
            y = (h * C[i][:, None, :]).sum(-1) + p["D"][:, None] * t["x"][i]
            loss = loss + (y * t["dy"][i]).sum()
        loss = loss + (h * t["dstate"][s]).sum()
        at += n
    return dict(zip(NAMES.values(), torch.autograd.grad(loss, list(p.values()))))


@pytest.mark.parametrize("lens,H,P,G,N,io", [([320], 8, 16, 1, 32, "bf16"), ([100, 7, 200], 8, 20, 2, 24, "bf16"),
                                             ([256], 4, 80, 1, 16, "bf16"), ([320], 8, 16, 1, 32, "f32"),
                                             ([100, 7, 200], 8, 22, 2, 25, "f32"), ([200], 4, 16, 1, 150, "bf16")])
def test_float32_gradients_have_float32_errors(lens, H, P, G, N, io):
    mine, plain, size = ({k: 0.0 for k in NAMES.values()} for _ in range(3))
    for seed in range(70, 74):
        c = ref.heads_inputs(seed, lens, H, P, G, N, io)
        exact, f32, got = gradients(c, torch.float64), gradients(c, torch.float32), run_backward(c)
        for k in NAMES.values():
            mine[k] += float((got[k].cpu().double() - exact[k]).square().sum())
            plain[k] += float((f32[k].double() - exact[k]).square().sum())
            size[k] += float(exact[k].square().sum())
    for k in NAMES.values():
        log(f"  {k}: {(mine[k] / size[k]) ** 0.5:.2e}, float32 throughout {(plain[k] / size[k]) ** 0.5:.2e}")
        assert mine[k] <= 9 * plain[k], k


def relative(got, want):
    return float((got.double().cpu() - want).norm() / want.norm())


@pytest.mark.parametrize("lens,H,P,G,N", [([300], 8, 16, 1, 32), ([5, 74, 37, 100], 8, 64, 2, 100), ([3] * 150 + [70], 7, 64, 1, 64)])
def test_bfloat16_gradients(lens, H, P, G, N):
    """dx and dB without initial states and final gradients, where nothing rounded but M meets them: their errors are those of
    one rounding of the result (at most 1.15 times, as the other operand's second part leaves 2^-17)."""
    c = ref.heads_inputs(75, lens, H, P, G, N, "bf16", state=False)
    c["dstate"].zero_()
    want, got = ref.backward(c), run_backward(c)
    for k in ("dx", "dB"):
        exact = want[k][0]
        once = relative(exact.to(torch.bfloat16), exact)
        mine = relative(got[k], exact)
        log(f"  {k}: {mine:.2e}, rounded once {once:.2e}")
        assert mine <= 1.15 * once, k
