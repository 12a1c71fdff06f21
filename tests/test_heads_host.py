"""The head scan's and the norms' calls without a GPU: bad arguments are refused on the host before anything is
enqueued, size queries, and the binding's own checks; the 64-bit reference against differences."""
from __future__ import annotations

import ctypes

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import heads_ref as ref

NULL, DIM, UNSUPPORTED, ALIGN, WORKSPACE, ALIAS = -1, -2, -3, -4, -5, -6
A, STEP = 0x10000000, 0x10000000  # fake, well aligned device addresses: refused before they are touched


@pytest.fixture(scope="module")
def lib():
    return mm.load()


def ptrs(n):
    return [ctypes.c_void_p(A + i * STEP) for i in range(n)]


def at(p, i, v):
    q = list(p)
    q[i] = ctypes.c_void_p(v)
    return q


def prefill(lib, p, S=2, T=5000, H=4, P=64, G=2, N=128, io=1, xs=256, ds=4, bs=256, cs=256, ws=0x7F0000000, wsb=1 << 40):
    return lib.mamba_mixer_heads_prefill(*p, S, T, H, P, G, N, io, xs, ds, bs, cs, ctypes.c_void_p(ws), wsb, None)


def decode(lib, p, Bs=2, H=4, P=64, G=2, N=128, io=1, xs=256, ds=4, bs=256, cs=256):
    return lib.mamba_mixer_heads_decode(*p, Bs, H, P, G, N, io, xs, ds, bs, cs, None)


def backward(lib, p, S=2, T=5000, H=4, P=64, G=2, N=128, io=1, xs=256, ds=4, bs=256, cs=256, gx=256, gd=4, gb=256, gc=256,
             ws=0x7F00000000, wsb=1 << 40):
    return lib.mamba_mixer_heads_backward(*p, S, T, H, P, G, N, io, xs, ds, bs, cs, gx, gd, gb, gc, ctypes.c_void_p(ws), wsb,
                                          None)


@pytest.mark.parametrize("call,n,optional", [(prefill, 11, (1, 5, 8)), (decode, 10, (1, 5, 7)),
                                             (backward, 19, (1, 5, 8, 10, 18))])
def test_heads_refusals(lib, call, n, optional):
    p = ptrs(n)
    for kw in (dict(io=2), dict(P=0), dict(P=257), dict(N=0), dict(N=257)):
        assert call(lib, p, **kw) == UNSUPPORTED, kw
    for kw in (dict(H=-1), dict(G=0), dict(G=3), dict(xs=255), dict(ds=3), dict(bs=255), dict(cs=1), dict(xs=-256)):
        assert call(lib, p, **kw) == DIM, kw
    if call is not decode:
        for kw in (dict(S=-1), dict(T=-1), dict(S=0), dict(T=2 ** 31)):
            assert call(lib, p, **kw) == DIM, kw
        assert call(lib, p, wsb=16) == WORKSPACE and call(lib, p, ws=0) == WORKSPACE
        assert call(lib, p, ws=0x7F00000010) == ALIGN
    if call is backward:
        for kw in (dict(gx=255), dict(gd=3), dict(gb=255), dict(gc=255)):
            assert call(lib, p, **kw) == DIM, kw
    for i in range(n):
        if i not in optional:
            assert call(lib, at(p, i, 0)) == NULL, i
        assert call(lib, at(p, i, p[i].value + 1)) == ALIGN, i
    first_out = {prefill: 9, decode: 8, backward: 11}[call]
    for o in range(first_out, n):
        for i in (0, 2, 3, 4):
            assert call(lib, at(p, o, p[i].value)) == ALIAS, (o, i)
        for k in range(first_out, o):
            assert call(lib, at(p, o, p[k].value)) == ALIAS, (o, k)
    if call is not backward:  # state_out may be state_in, but not overlap it otherwise
        state_in = {prefill: 8, decode: 7}[call]
        state_out = {prefill: 9, decode: 8}[call]
        assert call(lib, at(p, state_out, p[state_in].value + 4)) == ALIAS
    assert call(lib, [ctypes.c_void_p(0)] * n, H=0) == 0


def test_column_ranges_of_one_gradient_are_taken_apart(lib):
    p = ptrs(19)
    base = p[11].value  # dx | dB | dC | ddt in rows of 256 + 256 + 256 + 4 bfloat16 values
    row = 772
    apart = dict(gx=row, gd=row, gb=row, gc=row, wsb=0)
    p = at(at(at(p, 13, base + 512), 14, base + 1024), 12, base + 1536)
    assert backward(lib, p, **apart) == WORKSPACE  # past the overlap checks
    assert backward(lib, at(p, 13, base + 510), **apart) == ALIAS
    assert backward(lib, at(p, 12, base + 1536 + 2), **apart) == ALIAS  # wraps into the next row's dx
    assert backward(lib, p, **dict(apart, gb=row + 1)) == ALIAS


def test_workspace_queries(lib):
    q = lib.mamba_mixer_heads_prefill_workspace_bytes
    assert q(0, 0, 4, 64, 1, 128, 1) == 0 and q(1, 0, 4, 64, 1, 128, 1) == 0
    assert q(1, 64, 64, 64, 1, 128, 1) == 0
    assert q(1, 32768, 4, 64, 1, 128, 1) > 0
    assert q(1, 64, 4, 300, 1, 128, 1) == 0
    b = lib.mamba_mixer_heads_backward_workspace_bytes
    assert b(1, 4096, 4, 64, 1, 128, 1) > b(1, 64, 4, 64, 1, 128, 1) > 0
    assert lib.mamba_mixer_gate_norm_backward_workspace_bytes(4, 60, 7) == 0
    assert lib.mamba_mixer_gate_norm_backward_workspace_bytes(4, 64, 1) > 0
    assert lib.mamba_mixer_residual_norm_backward_workspace_bytes(4, 1 << 20) == 0


def gate(lib, p, rows=4, d=64, g=1, eps=1e-5, io=1, ys=64, zs=64):
    return lib.mamba_mixer_gate_norm(*p, rows, d, g, eps, 1, io, ys, zs, None)


def gate_backward(lib, p, rows=4, d=64, g=1, eps=1e-5, io=1, ys=64, zs=64, gy=64, gz=64, ws=0x7F00000000, wsb=1 << 30):
    return lib.mamba_mixer_gate_norm_backward(*p, rows, d, g, eps, 1, io, ys, zs, gy, gz, ctypes.c_void_p(ws), wsb, None)


def test_gate_norm_refusals(lib):
    for call, n in ((gate, 4), (gate_backward, 7)):
        p = ptrs(n)
        for kw in (dict(rows=-1), dict(d=-1), dict(g=0), dict(g=3), dict(eps=-1.0), dict(eps=float("nan")), dict(ys=63),
                   dict(zs=63)):
            assert call(lib, p, **kw) == DIM, kw
        assert call(lib, p, io=7) == UNSUPPORTED
        for i in range(n):
            assert call(lib, at(p, i, 0)) == NULL, i
            assert call(lib, at(p, i, p[i].value + 1)) == ALIGN, i
    p = ptrs(4)
    assert gate(lib, at(p, 3, p[1].value)) == ALIAS and gate(lib, at(p, 3, p[0].value + 2)) == ALIAS
    assert gate(lib, at(p, 3, p[0].value), ys=128) == ALIAS
    assert gate(lib, [ctypes.c_void_p(0)] * 4, rows=0) == 0
    p = ptrs(7)
    for o in (4, 5, 6):
        for i in range(o):
            assert gate_backward(lib, at(p, o, p[i].value)) == ALIAS, (o, i)
    assert gate_backward(lib, p, wsb=8) == WORKSPACE and gate_backward(lib, p, ws=8) == ALIGN
    q = at(p, 5, p[4].value + 128)  # dy | dz in rows of 128
    assert gate_backward(lib, q, gy=128, gz=128, wsb=8) == WORKSPACE
    assert gate_backward(lib, q, gy=128, gz=130, wsb=8) == ALIAS


def residual(lib, p, rows=4, d=64, eps=1e-5, io=1, res=0):
    return lib.mamba_mixer_residual_norm(*p[:5], 1.0, *p[5:], rows, d, eps, io, res, None)


def residual_backward(lib, p, rows=4, d=64, eps=1e-5, io=1, res=0, ws=0x7F00000000, wsb=1 << 30):
    return lib.mamba_mixer_residual_norm_backward(*p[:7], 1.0, *p[7:], rows, d, eps, io, res, ctypes.c_void_p(ws), wsb, None)


def test_residual_norm_refusals(lib):
    for call, n, optional in ((residual, 7, (1, 3, 4)), (residual_backward, 12, (1, 5, 6))):
        p = ptrs(n)
        for kw in (dict(rows=-1), dict(d=-1), dict(eps=-1.0)):
            assert call(lib, p, **kw) == DIM, kw
        for kw in (dict(io=7), dict(res=3), dict(io=0, res=1), dict(d=32769)):
            assert call(lib, p, **kw) == UNSUPPORTED, kw
        for i in range(n):
            if i not in optional:
                assert call(lib, at(p, i, 0)) == NULL, i
            assert call(lib, at(p, i, p[i].value + 1)) == ALIGN, i
    p = ptrs(7)
    assert residual(lib, at(p, 6, p[0].value)) == ALIAS and residual(lib, at(p, 6, p[5].value)) == ALIAS
    assert residual(lib, at(p, 6, p[1].value)) == ALIAS and residual(lib, at(p, 5, p[1].value + 4)) == ALIAS
    assert residual(lib, [ctypes.c_void_p(0)] * 7, rows=0) == 0
    p = ptrs(12)
    assert residual_backward(lib, p, wsb=8) == WORKSPACE and residual_backward(lib, p, ws=8) == ALIGN
    assert residual_backward(lib, at(p, 7, p[3].value)) == ALIAS and residual_backward(lib, at(p, 9, p[10].value)) == ALIAS


def test_binding_checks():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    f = torch.float32
    ok = dict(x=t(5, 4, 8), dt=t(5, 4), B=t(5, 2, 16), C=t(5, 2, 16), A_log=t(4, dtype=f), D=t(4, dtype=f),
              dt_bias=t(4, dtype=f))
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        mm.heads_prefill(**ok, cu_seqlens=cu)
    for k, v, err in (("x", t(5, 4), ValueError), ("x", t(5, 4, 8, dtype=torch.float16), TypeError),
                      ("B", t(5, 32), ValueError)):
        with pytest.raises(err):
            mm.heads_prefill(**dict(ok, **{k: v}), cu_seqlens=cu)
    with pytest.raises(ValueError):
        mm.gate_norm(t(3), t(3), t(3, dtype=f))
    with pytest.raises(ValueError):
        mm.residual_norm(t(3), t(3), t(3, dtype=f))


def test_reference_gradients_against_differences():
    """The 64-bit adjoint that the GPU gradients are compared with, along random directions."""
    c = ref.heads_inputs(15, [9, 0, 20], 4, 5, 2, 3, "f32")
    want = ref.backward(c)
    for k, gk in dict(x="dx", dt="ddt", B="dB", C="dC", A_log="dA_log", D="dD", dt_bias="ddt_bias", state="dstate_in").items():
        v = torch.randn(c[k].shape, generator=torch.Generator().manual_seed(3), dtype=torch.float64)
        loss = []
        for e in (1e-5, -1e-5):
            d = dict(c)
            d[k] = c[k].double() + e * v
            y, s, _, _ = ref.forward(d)
            loss.append(float((y * c["dy"].double()).sum() + (s * c["dstate"].double()).sum()))
        diff, mine = (loss[0] - loss[1]) / 2e-5, float((want[gk][0] * v).sum())
        assert abs(mine - diff) <= 1e-6 * (1 + abs(mine)), k
