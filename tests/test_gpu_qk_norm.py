"""The norms of queries and keys with their rotation against their definition in 64 bits.  Needs an MI355X."""
from __future__ import annotations

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu

# T, Hq, Hk, D, R, io
CASES = [(1, 1, 1, 2, 2, "f32"), (1, 8, 8, 128, 128, "bf16"), (5, 3, 1, 64, 32, "bf16"), (33, 4, 2, 40, 40, "f32"),
         (7, 2, 2, 1, 0, "f32"), (100, 8, 1, 50, 26, "bf16"), (64, 1, 1, 256, 256, "bf16"), (19, 5, 5, 80, 0, "bf16"),
         (300, 6, 2, 96, 96, "f32"), (12, 2, 3, 255, 254, "f32"), (2050, 3, 3, 64, 64, "bf16"), (40, 24, 8, 16, 4, "bf16"),
         (9, 2, 2, 192, 64, "bf16"), (513, 1, 2, 20, 10, "bf16")]


def gpu(t):
    return t.cuda() if t is not None else None


def strided(c):
    T, Hq, D = c["q"].shape
    Hk = c["k"].shape[1]
    p = torch.zeros(T, (Hq + Hk) * D + 3, dtype=c["q"].dtype, device="cuda")
    q, k = p[:, :Hq * D].unflatten(1, (Hq, D)), p[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    q.copy_(c["q"])
    k.copy_(c["k"])
    return q, k


def call(c, q, k, inter, **kw):
    return mm.qk_norm(q, k, c["wq"].cuda(), c["wk"].cuda(), gpu(c["pos"]), gpu(c["freq"]), interleaved=inter, **kw)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R,io", CASES)
def test_forward(T, Hq, Hk, D, R, io, inter):
    c = ref.qk_inputs(1, T, Hq, Hk, D, R, io)
    q, k = strided(c)
    got = call(c, q, k, inter)
    for g, (w, mag), n in zip(got, ref.qk(c, inter), "qk"):
        ref.check(g, w, mag, D, n)
    dense = call(c, c["q"].cuda().contiguous(), c["k"].cuda().contiguous(), inter)
    same = call(c, q, k, inter, q_out=q, k_out=k)
    assert same[0] is q and same[1] is k
    for g, e, s in zip(got, dense, same):
        assert torch.equal(g, e) and torch.equal(g, s), "dense rows, in place"


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R,io", CASES)
def test_backward(T, Hq, Hk, D, R, io, inter):
    c = ref.qk_inputs(2, T, Hq, Hk, D, R, io)
    q, k = strided(c)
    out = torch.full((T, (Hq + Hk) * D + 1), ref.NAN, dtype=c["q"].dtype, device="cuda")
    dq, dk = out[:, :Hq * D].unflatten(1, (Hq, D)), out[:, Hq * D:-1].unflatten(1, (Hk, D))
    run = lambda **kw: mm.qk_norm_backward(c["dq"].cuda(), c["dk"].cuda(), q, k, c["wq"].cuda(), c["wk"].cuda(), gpu(c["pos"]),  # noqa: E731
                                           gpu(c["freq"]), interleaved=inter, **kw)
    got = run(dq=dq, dk=dk)
    assert out[:, -1].isnan().all()
    want = ref.qk_backward(c, inter)
    for g, n in zip(got, ("dq", "dk", "dwq", "dwk")):
        v, mag = want[n]
        ref.check(g, v, mag, T * max(Hq, Hk) if n[1] == "w" else D, n)
    for a, b in zip(run(), got):
        assert torch.equal(a, b), "a call repeats bit for bit"


@pytest.mark.parametrize("pos", [2 ** 31 - 1, -2 ** 31, -5, 0, 123456789])
def test_far_positions(pos):
    c = ref.qk_inputs(3, 4, 2, 2, 64, 64, "f32")
    c["pos"] = torch.full((4,), pos, dtype=torch.int32)
    for g, (w, mag), n in zip(call(c, c["q"].cuda(), c["k"].cuda(), False), ref.qk(c, False), "qk"):
        ref.check(g, w, mag, 64, n)


def test_rows_of_zeros_and_values_that_are_not_finite():
    c = ref.qk_inputs(4, 20, 3, 2, 64, 32, "bf16")
    q, k = c["q"].cuda().contiguous(), c["k"].cuda().contiguous()
    clean = call(c, q, k, True)
    q[3, 1] = 0
    k[7, 0, 5] = ref.NAN
    k[9, 1, 50] = float("inf")
    a, b = call(c, q, k, True)
    assert not a[3, 1].any() and b[7, 0].isnan().all()
    assert b[9, 1, 50].isnan() and not b[9, 1, 40].any()  # n(v) of an infinite row: inf / inf, and 0 elsewhere
    keep = torch.ones(20, 2, dtype=torch.bool, device="cuda")
    keep[7, 0] = keep[9, 1] = False
    assert torch.equal(b[keep], clean[1][keep])
    back = mm.qk_norm_backward(c["dq"].cuda(), c["dk"].cuda(), q, k, c["wq"].cuda(), c["wk"].cuda(), gpu(c["pos"]), gpu(c["freq"]),
                               interleaved=True)
    assert back[0].isfinite().all() and back[2].isfinite().all() and back[1][keep].isfinite().all()
    assert back[1][7, 0].isnan().all() and back[3].isnan().all()


def test_empty_calls():
    q, w = torch.zeros(0, 2, 8, device="cuda"), torch.ones(8, device="cuda")
    assert [t.shape[0] for t in mm.qk_norm(q, q, w, w)] == [0, 0]
    got = mm.qk_norm_backward(q, q, q, q, w, w)
    assert not got[2].any() and not got[3].any()


@pytest.mark.parametrize("T,Hq,Hk,D,R,io", [(9001, 2, 1, 32, 16, "bf16"), (70001, 1, 2, 6, 4, "f32"), (2501, 5, 3, 36, 20, "bf16")])
def test_more_tokens_than_workgroups(T, Hq, Hk, D, R, io):
    c = ref.qk_inputs(5, T, Hq, Hk, D, R, io)
    q, k = strided(c)
    for g, (w, mag), n in zip(call(c, q, k, False), ref.qk(c, False), "qk"):
        ref.check(g, w, mag, D, n)
    got = mm.qk_norm_backward(c["dq"].cuda(), c["dk"].cuda(), q, k, c["wq"].cuda(), c["wk"].cuda(), gpu(c["pos"]), gpu(c["freq"]))
    want = ref.qk_backward(c, False)
    for g, n in zip(got, ("dq", "dk", "dwq", "dwk")):
        v, mag = want[n]
        ref.check(g, v, mag, T * max(Hq, Hk) if n[1] == "w" else D, n)
