"""The gated norm and the residual norm against their definitions in 64 bits; the gradients against torch's
differentiation of those and against differences.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import heads_ref as ref

pytestmark = pytest.mark.gpu

DT = dict(bf16=torch.bfloat16, f32=torch.float32)
GATE = [(1, 64, 1, "bf16"), (3, 7, 1, "f32"), (5, 4096, 1, "bf16"), (33, 40, 8, "bf16"), (300, 1, 1, "f32"),
        (17, 5120, 8, "bf16"), (9, 2049, 1, "bf16"), (4, 16384, 2, "f32"), (2, 40000, 1, "bf16"), (600, 1536, 1, "bf16"),
        (257, 130, 2, "f32")]
RES = [(1, 2048, "bf16", "f32"), (3, 7, "f32", "f32"), (70, 2560, "bf16", "f32"), (5, 2049, "bf16", "bf16"),
       (300, 1, "f32", "f32"), (2, 32768, "bf16", "f32"), (513, 768, "bf16", "bf16"), (40, 4100, "f32", "f32")]


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def gate_case(rows, d, io):
    y, z, do = (rnd(s, rows, d).to(DT[io]) for s in (1, 2, 3))
    wide = torch.zeros(rows, 2 * d, dtype=DT[io])
    wide[:, d:] = z
    return y, z, do, 1 + 0.1 * rnd(4, d), wide.cuda()[:, d:]


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("rows,d,groups,io", GATE)
def test_gate_norm(rows, d, groups, io, gate_first):
    y, z, do, w, zs = gate_case(rows, d, io)
    out = mm.gate_norm(y.cuda(), zs, w.cuda(), groups=groups, gate_first=gate_first)
    r = ref.gate_norm(y.double(), z.double(), w.double(), groups, gate_first)
    ref.check_rows(out, r, r.abs(), "out")
    yc = y.cuda()
    assert mm.gate_norm(yc, zs, w.cuda(), groups=groups, gate_first=gate_first, out=yc) is yc
    assert torch.equal(yc, out), "in place"


def row_max(v, groups):
    """The largest magnitude of each (row, group), at every element of it: a bound of the mean that is subtracted."""
    return v.abs().reshape(v.shape[0], groups, -1).amax(2, keepdim=True).expand(-1, -1, v.shape[1] // groups).reshape(v.shape)


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("rows,d,groups,io", GATE)
def test_gate_norm_backward(rows, d, groups, io, gate_first):
    y, z, do, w, zs = gate_case(rows, d, io)
    both = torch.zeros(rows, 2 * d, dtype=DT[io], device="cuda")  # the gradient of [z | y]
    dy, dz, dw = mm.gate_norm_backward(do.cuda(), y.cuda(), zs, w.cuda(), groups=groups, gate_first=gate_first,
                                       dz=both[:, :d], dy=both[:, d:])
    leaves = [t.double().requires_grad_(True) for t in (y, z, w)]
    want = torch.autograd.grad(ref.gate_norm(*leaves, groups, gate_first), leaves, do.double())
    # dy and dz are differences of the direct term and the mean's: the row's largest values bound both
    terms = [row_max(t, groups) + 0 * t for t in want[:2]]
    u = (y.double() * z.double() * torch.sigmoid(z.double())) if gate_first else y.double()
    k = 1 / torch.sqrt((u.reshape(rows, groups, -1) ** 2).mean(2, keepdim=True) + ref.EPS)
    scale = k.expand(-1, -1, d // groups).reshape(rows, d) * row_max(do.double() * w.double() * (1 + z.double().abs()), groups)
    terms = [t + scale * (1 + z.double().abs()) * (1 + (y.double().abs() if i else 0)) for i, t in enumerate(terms)]
    ref.check_rows(dy, want[0], terms[0], "dy")
    ref.check_rows(dz, want[1], terms[1], "dz")
    each = (do.double() * ref.gate_norm(y.double(), z.double(), torch.ones(d, dtype=torch.float64), groups, gate_first)).abs()
    ref.check_rows(dw, want[2], each.sum(0), "dweight")


def res_case(rows, d, io, res, post, vec):
    h, do = rnd(1, rows, d).to(DT[io]), rnd(2, rows, d).to(DT[io])
    r, dr = 3 * rnd(3, rows, d).to(DT[res]), rnd(4, rows, d).to(DT[res])
    w, wp, v = (1 + 0.1 * rnd(s, d) for s in (5, 6, 7))
    return h, do, r.to(DT[res]), dr, w, wp if post else None, v if vec else None


def cuda(t):
    return t.cuda() if t is not None else None


def dbl(t):
    return t.double() if t is not None else None


@pytest.mark.parametrize("post,vec", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows,d,io,res", RES)
def test_residual_norm(rows, d, io, res, post, vec):
    h, _, r, _, w, wp, v = res_case(rows, d, io, res, post, vec)
    kw = dict(post_weight=cuda(wp), scale=0.5, scale_vec=cuda(v))
    out, new = mm.residual_norm(h.cuda(), r.cuda(), w.cuda(), **kw)
    ro, rn = ref.residual_norm(dbl(h), dbl(r), dbl(w), dbl(wp), 0.5, dbl(v))
    mag = dbl(r).abs() + (rn - dbl(r)).abs()
    ref.check_rows(new, rn, mag, "residual")
    k = (1 / torch.sqrt((rn ** 2).mean(1, keepdim=True) + ref.EPS))
    ref.check_rows(out, ro, ro.abs() + mag * k * dbl(w).abs(), "out")
    rc = r.cuda()
    assert mm.residual_norm(h.cuda(), rc, w.cuda(), residual_out=rc, **kw)[1] is rc
    assert torch.equal(rc, new), "in place"


def test_residual_norm_without_a_residual():
    h, _, _, _, w, wp, v = res_case(5, 96, "bf16", "bf16", True, True)
    out, new = mm.residual_norm(h.cuda(), None, w.cuda(), post_weight=wp.cuda(), scale_vec=v.cuda())
    o2, n2 = mm.residual_norm(h.cuda(), torch.zeros_like(h).cuda(), w.cuda(), post_weight=wp.cuda(), scale_vec=v.cuda())
    assert torch.equal(out, o2) and torch.equal(new, n2)


@pytest.mark.parametrize("post,vec", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows,d,io,res", RES)
def test_residual_norm_backward(rows, d, io, res, post, vec):
    h, do, r, dr, w, wp, v = res_case(rows, d, io, res, post, vec)
    kw = dict(post_weight=cuda(wp), scale=0.5, scale_vec=cuda(v))
    for upstream in (dr, None):
        got = mm.residual_norm_backward(do.cuda(), cuda(upstream), h.cuda(), r.cuda(), w.cuda(), **kw)
        R, W = (t.double().requires_grad_(True) for t in (r, w))
        dR, dW = torch.autograd.grad(ref._norm(R) * W, (R, W), do.double())
        k = 1 / torch.sqrt((dbl(r) ** 2).mean(1, keepdim=True) + ref.EPS)
        mag_R = row_max(do.double() * dbl(w), 1) * k * (1 + dbl(r).abs() * k) + (dbl(dr).abs() if upstream is not None else 0)
        dR = dR + (dbl(upstream) if upstream is not None else 0)
        leaves = {"dh": dbl(h).requires_grad_(True)}
        if post:
            leaves["dpost_weight"] = dbl(wp).requires_grad_(True)
        if vec:
            leaves["dscale_vec"] = dbl(v).requires_grad_(True)
        n = ref._norm(leaves["dh"]) if post else leaves["dh"]
        p = n * leaves["dpost_weight"] if post else n
        change = 0.5 * p * (leaves["dscale_vec"] if vec else 1.0)
        want = dict(zip(leaves, torch.autograd.grad(change, list(leaves.values()), dR)))
        ref.check_rows(got["dresidual"], dR, mag_R, "dresidual")
        ref.check_rows(got["dweight"], dW, (do.double() * dbl(r) * k).abs().sum(0), "dweight")
        kp = 1 / torch.sqrt((dbl(h) ** 2).mean(1, keepdim=True) + ref.EPS) if post else 1.0
        f = 0.5 * (dbl(v).abs() if vec else 1.0) * (dbl(wp).abs() if post else 1.0)
        big = row_max(mag_R * f, 1) * kp
        ref.check_rows(got["dh"], want["dh"], big * (1 + dbl(h).abs() * kp) if post else mag_R * f, "dh")
        if post:
            ref.check_rows(got["dpost_weight"], want["dpost_weight"],
                           (mag_R * 0.5 * (dbl(v).abs() if vec else 1.0) * (n.detach()).abs()).sum(0), "dpost_weight")
        if vec:
            ref.check_rows(got["dscale_vec"], want["dscale_vec"], (mag_R * 0.5 * p.detach().abs()).sum(0), "dscale_vec")
        assert set(got) == {"dresidual", "dweight", *want}
    inplace = dr.cuda()
    again = mm.residual_norm_backward(do.cuda(), inplace, h.cuda(), r.cuda(), w.cuda(), dresidual=inplace, **kw)
    first = mm.residual_norm_backward(do.cuda(), dr.cuda(), h.cuda(), r.cuda(), w.cuda(), **kw)
    for key in first:
        assert torch.equal(again[key], first[key]), f"{key}: in place"


def test_gradients_against_differences():
    """Along a direction, against central differences of the 64-bit definitions (step 1e-4)."""
    rows, d, groups = 6, 48, 4
    y, z, do, w, zs = gate_case(rows, d, "f32")
    for first in (True, False):
        got = mm.gate_norm_backward(do.cuda(), y.cuda(), zs, w.cuda(), groups=groups, gate_first=first)
        for i, g in enumerate(got):
            args = [dbl(y), dbl(z), dbl(w)]
            v = rnd(20 + i, *g.shape).double()
            f = [float((ref.gate_norm(*[a + e * v if j == i else a for j, a in enumerate(args)], groups, first) * dbl(do)).sum())
                 for e in (1e-4, -1e-4)]
            mine, diff = float((g.cpu().double() * v).sum()), (f[0] - f[1]) / 2e-4
            assert abs(mine - diff) <= 1e-4 * float((g.cpu().double() * v).abs().sum()), (first, i)


@pytest.mark.parametrize("scale", [0.0, 1e-20, 1e15])
def test_rows_of_zeros_and_extreme_sizes(scale):
    """eps alone keeps a row of zeros finite; tiny and large rows stay finite in float32."""
    y = scale * rnd(1, 3, 256)
    z = rnd(2, 3, 256)
    w = torch.ones(256)
    out = mm.gate_norm(y.cuda(), z.cuda(), w.cuda())
    r = ref.gate_norm(dbl(y), dbl(z), dbl(w), 1, True)
    ref.check_rows(out, r, r.abs() + 1e-20, "out")
    o, n = mm.residual_norm(y.cuda(), torch.zeros(3, 256).cuda(), w.cuda())
    ro, _ = ref.residual_norm(dbl(y), torch.zeros(3, 256).double(), dbl(w), None, 1.0, None)
    ref.check_rows(o, ro, ro.abs() + 1e-20, "out")
