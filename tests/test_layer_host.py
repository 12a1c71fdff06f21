"""The convolution's, the gated recurrence's and the head norm's calls without a GPU: bad arguments are refused on the host
before anything is enqueued, in-place pairs, size queries, the binding's own checks and its streams; the 64-bit references
against differences."""
from __future__ import annotations

import ctypes

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import layer_ref as ref
from tests import test_binding_streams as streams
from tests.test_binding_streams import CURRENT, SIDE, cu, dev, recorded  # noqa: F401

NULL, DIM, UNSUPPORTED, ALIGN, WORKSPACE, ALIAS = -1, -2, -3, -4, -5, -6
A, STEP = 0x10000000, 0x10000000  # fake, well aligned device addresses: refused before they are touched
WS = 0x7F00000000


@pytest.fixture(scope="module")
def lib():
    return mm.load()


def ptrs(n, step=STEP):
    return [ctypes.c_void_p(A + i * step) for i in range(n)]


def at(p, i, v):
    q = list(p)
    q[i] = ctypes.c_void_p(v)
    return q


def conv(lib, p, S=2, T=500, d=64, W=4, io=1, xs=64):
    return lib.mamba_mixer_conv_prefill(*p, S, T, d, W, 1, io, xs, None)


def conv_decode(lib, p, S=2, d=64, W=4, io=1, xs=64):
    return lib.mamba_mixer_conv_decode(*p, S, d, W, 1, io, xs, None)


def conv_backward(lib, p, S=2, T=500, d=64, W=4, io=1, xs=64, gx=64, ws=WS, wsb=1 << 40):
    return lib.mamba_mixer_conv_backward(*p, S, T, d, W, 1, io, xs, gx, ctypes.c_void_p(ws), wsb, None)


def gated(lib, p, S=2, T=5000, d=64, c=8.0, gate=0, io=1, xs=64, rs=64, gs=64, zs=64, ws=WS, wsb=1 << 40):
    return lib.mamba_mixer_gated_prefill(*p, S, T, d, c, gate, io, xs, rs, gs, zs, ctypes.c_void_p(ws), wsb, None)


def gated_decode(lib, p, S=2, d=64, c=8.0, gate=0, io=1, xs=64, rs=64, gs=64, zs=64):
    return lib.mamba_mixer_gated_decode(*p, S, d, c, gate, io, xs, rs, gs, zs, None)


def gated_backward(lib, p, S=2, T=5000, d=64, c=8.0, gate=0, io=1, xs=64, rs=64, gs=64, zs=64, dxs=64, drs=64, dgs=64, dzs=64,
                   ws=WS, wsb=1 << 40):
    return lib.mamba_mixer_gated_backward(*p, S, T, d, c, gate, io, xs, rs, gs, zs, dxs, drs, dgs, dzs, ctypes.c_void_p(ws), wsb,
                                          None)


def qk(lib, p, T=500, Hq=4, Hk=2, D=64, R=32, eps=1e-5, io=1, qs=256, ks=128, qos=256, kos=128):
    return lib.mamba_mixer_qk_norm(*p, T, Hq, Hk, D, R, eps, 0, io, qs, ks, qos, kos, None)


def qk_backward(lib, p, T=500, Hq=4, Hk=2, D=64, R=32, eps=1e-5, io=1, qs=256, ks=128, dqs=256, dks=128, ws=WS, wsb=1 << 40):
    return lib.mamba_mixer_qk_norm_backward(*p, T, Hq, Hk, D, R, eps, 0, io, qs, ks, dqs, dks, ctypes.c_void_p(ws), wsb, None)


# call, its pointers, the optional ones, the first output, outputs that are needed only with an optional input {out: in}
CALLS = {
    conv: (7, (2, 4), 5, {}), conv_decode: (6, (2, 3), 4, {}), conv_backward: (11, (2, 4, 6, 10), 7, {9: 2}),
    gated: (10, (2, 3, 4, 6, 9), 7, {}), gated_decode: (8, (2, 3, 4, 5), 6, {}),
    gated_backward: (16, (2, 3, 4, 6, 8, 9, 15), 10, {12: 2, 13: 3, 14: 4}), qk: (8, (), 6, {}), qk_backward: (12, (), 8, {}),
}
IN_PLACE = {conv: {(5, 4)}, conv_decode: {(4, 3)}, gated: {(7, 6)}, gated_decode: {(6, 5)}, qk: {(6, 0), (7, 1)}}


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_refusals(lib, call):
    n, optional, first_out, needs = CALLS[call]
    p = ptrs(n)
    assert call(lib, p, io=2) == UNSUPPORTED
    sizes = [dict(xs=63)] if call not in (qk, qk_backward) else [dict(qs=255), dict(ks=127), dict(Hq=0), dict(Hk=0), dict(R=31),
                                                                  dict(R=66), dict(R=-2), dict(eps=-1.0), dict(eps=float("nan")),
                                                                  dict(T=-1), dict(T=2 ** 31 // 6 + 1)]
    if call in (gated, gated_decode, gated_backward):
        sizes += [dict(rs=63), dict(gs=63), dict(zs=0), dict(c=-1.0), dict(c=float("nan")), dict(c=float("inf"))]
        assert call(lib, p, gate=2) == UNSUPPORTED and call(lib, p, gate=-1) == UNSUPPORTED
    if call in (conv, conv_decode, conv_backward):
        assert call(lib, p, W=1) == UNSUPPORTED and call(lib, p, W=5) == UNSUPPORTED
    if call not in (qk, qk_backward):
        sizes += [dict(S=-1), dict(d=-1), dict(S=2 ** 26)]
        if call not in (conv_decode, gated_decode):
            sizes += [dict(T=-1), dict(T=2 ** 31), dict(S=0)]
    if call is gated_backward:
        sizes += [dict(dxs=63), dict(drs=-64), dict(dgs=63), dict(dzs=63)]
    if call is conv_backward:
        sizes += [dict(gx=63)]
    if call is qk:
        sizes += [dict(qos=255), dict(kos=127)]
    if call is qk_backward:
        sizes += [dict(dqs=255), dict(dks=127)]
    for kw in sizes:
        assert call(lib, p, **kw) == DIM, kw
    if call in (qk, qk_backward):
        assert call(lib, p, D=257) == UNSUPPORTED and call(lib, p, D=0, R=0) == UNSUPPORTED
    if call in (conv_backward, gated_backward, qk_backward):
        assert call(lib, p, wsb=16) == WORKSPACE and call(lib, p, ws=0) == WORKSPACE and call(lib, p, ws=WS + 16) == ALIGN
    for i in range(n):
        if i not in optional:
            assert call(lib, at(p, i, 0)) == NULL, i
        assert call(lib, at(p, i, p[i].value + 1)) == ALIGN, i
    for o in range(first_out, n):
        for i in range(n):
            if i == o or (o, i) in IN_PLACE.get(call, ()) or (i, o) in IN_PLACE.get(call, ()):
                continue
            assert call(lib, at(p, o, p[i].value)) == ALIAS, (o, i)
    for o, i in IN_PLACE.get(call, ()):
        assert call(lib, at(p, o, p[i].value + 4)) == ALIAS, "an input's middle"
        q = at(p, o, p[i].value)
        for k in range(n):
            if k not in (o, i):
                assert call(lib, at(q, k, p[i].value)) == ALIAS, ("a third array at the in-place address", o, i, k)


def test_in_place_needs_the_same_rows(lib):
    p = ptrs(8)
    assert qk(lib, at(p, 6, p[0].value), qs=256, qos=260) == ALIAS
    assert qk(lib, at(p, 7, p[1].value), ks=130, kos=128) == ALIAS


def test_column_ranges_of_one_array_are_taken_apart(lib):
    p = ptrs(16)
    base = p[10].value  # dx | dr | dg | dz in rows of 256 bfloat16 values
    row = dict(dxs=256, drs=256, dgs=256, dzs=256, wsb=0)
    q = at(at(at(p, 11, base + 128), 12, base + 256), 13, base + 384)
    assert gated_backward(lib, q, **row) == WORKSPACE  # past the overlap checks
    assert gated_backward(lib, at(q, 11, base + 126), **row) == ALIAS
    assert gated_backward(lib, q, **dict(row, dgs=260)) == ALIAS
    p = ptrs(12)
    q = at(p, 9, p[8].value + 512)  # dq | dk in rows of 384
    assert qk_backward(lib, q, dqs=384, dks=384, wsb=0) == WORKSPACE
    assert qk_backward(lib, q, dqs=384, dks=386, wsb=0) == ALIAS


def test_calls_of_no_size(lib):
    none = lambda n: [ctypes.c_void_p(0)] * n  # noqa: E731
    assert conv(lib, none(7), d=0, xs=0) == 0 and conv_decode(lib, none(6), S=0) == 0 and conv_backward(lib, none(11), d=0, xs=0, gx=0) == 0
    assert gated(lib, none(10), d=0) == 0 and gated_decode(lib, none(8), d=0) == 0 and gated_backward(lib, none(16), d=0) == 0
    assert qk(lib, none(8), T=0) == 0
    assert conv(lib, none(7), S=0, T=0) == NULL  # the weights are needed


def test_sizes_at_the_launches_limits(lib):
    far = lambda n: ptrs(n, 1 << 42)  # noqa: E731
    assert conv_backward(lib, far(11), T=2 ** 31 - 1, d=15, xs=15, gx=15, wsb=0) == WORKSPACE
    assert conv_backward(lib, far(11), T=2 ** 31 - 1, d=512, xs=512, gx=512, wsb=0) == DIM
    rows = lambda d: {k: d for k in ("d", "xs", "rs", "gs", "zs", "dxs", "drs", "dgs", "dzs")}  # noqa: E731
    assert gated_backward(lib, far(16), T=2 ** 29 - 128, wsb=0, **rows(32)) == WORKSPACE
    assert gated_backward(lib, far(16), T=2 ** 29, wsb=0, **rows(32)) == DIM
    wide = {k: 2 ** 22 + 1 for k in ("xs", "rs", "gs", "zs", "dxs", "drs", "dgs", "dzs")}
    for k, v in wide.items():
        assert gated_backward(lib, far(16), **{k: v}, wsb=0) == UNSUPPORTED, k
    assert gated(lib, far(10), zs=2 ** 22 + 1) == UNSUPPORTED and gated_decode(lib, far(8), rs=2 ** 22 + 1) == UNSUPPORTED
    assert gated(lib, far(10), zs=2 ** 22, wsb=0) == WORKSPACE
    assert qk_backward(lib, far(12), T=(2 ** 31 - 1) // 6, wsb=0) == WORKSPACE


def test_size_queries(lib):
    assert lib.mamba_mixer_conv_backward_workspace_bytes(4000, 64, 4) > lib.mamba_mixer_conv_backward_workspace_bytes(40, 64, 4) > 0
    assert lib.mamba_mixer_conv_backward_workspace_bytes(40, 64, 5) == 0 == lib.mamba_mixer_conv_backward_workspace_bytes(-1, 64, 4)
    assert lib.mamba_mixer_gated_checkpoint_bytes(65, 10) == 80 and lib.mamba_mixer_gated_checkpoint_bytes(-1, 10) == 0
    assert lib.mamba_mixer_gated_backward_workspace_bytes(1 << 20, 64, 0) >= lib.mamba_mixer_gated_backward_workspace_bytes(1 << 20, 64, 1) > 0
    assert lib.mamba_mixer_gated_prefill_workspace_bytes(1, 64) == 0
    assert lib.mamba_mixer_qk_norm_backward_workspace_bytes(10, 2, 2, 64) > 0 == lib.mamba_mixer_qk_norm_backward_workspace_bytes(10, 2, 2, 300)
    assert mm.layer.GATED_BLOCK == 64


def test_binding_checks():
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    f = torch.float32
    c2 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        mm.conv_prefill(t(5, 4), t(4, 4, dtype=f), None, c2)
    for bad in ((t(5), t(4, 4, dtype=f)), (t(5, 4), t(4, dtype=f))):
        with pytest.raises(ValueError):
            mm.conv_prefill(*bad, None, c2)
    with pytest.raises(TypeError):
        mm.conv_prefill(t(5, 4, dtype=torch.float16), t(4, 4, dtype=f), None, c2)
    with pytest.raises(ValueError, match="gate"):
        mm.gated_decode(t(5, 4), t(5, 4), None, t(5, 4), None, gate="relu")
    with pytest.raises(ValueError):
        mm.gated_prefill_train(t(5), t(5), None, None, None, c2)
    with pytest.raises(ValueError, match="both"):
        mm.qk_norm(t(5, 2, 8), t(5, 2, 8), t(8, dtype=f), t(8, dtype=f), positions=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError):
        mm.qk_norm(t(5, 8), t(5, 8), t(8, dtype=f), t(8, dtype=f))


def test_tensors_of_another_device_are_refused():
    class Elsewhere(streams.OnDevice):
        device = torch.device("cuda", 7)

        def get_device(self):
            return 7

    other = torch.zeros(3, 64, dtype=streams.BF16).as_subclass(Elsewhere)
    with pytest.raises(ValueError, match="cuda:7"):
        mm.gated_decode(dev(3, 64), other, None, None, None, stream=CURRENT)
    assert not streams.LOG.launched


# ------------------------------------------------------------------------------------------ streams
F32 = torch.float32


def b_conv_prefill(**kw):
    return mm.conv_prefill(dev(60, 64), dev(64, 4, dtype=F32), None, cu(60), **kw)


def b_conv_decode(**kw):
    return mm.conv_decode(dev(3, 64), dev(64, 4, dtype=F32), None, **kw)


def b_conv_backward(**kw):
    return mm.conv_backward(dev(60, 64), dev(64, 4, dtype=F32), dev(64, dtype=F32), cu(60), None, dev(60, 64), **kw).values()


def b_gated_prefill(**kw):
    return mm.gated_prefill(dev(6000, 64), dev(6000, 64), None, dev(6000, 64), dev(64, dtype=F32), cu(6000), **kw)


def b_gated_prefill_train(**kw):
    return mm.gated_prefill_train(dev(6000, 64), dev(6000, 64), None, dev(6000, 64), dev(64, dtype=F32), cu(6000), **kw)


def b_gated_decode(**kw):
    return mm.gated_decode(dev(3, 64), dev(3, 64), dev(3, 64), None, None, **kw)


def b_gated_backward(**kw):
    x = dev(6000, 64)
    return mm.gated_backward(x, x, x, x, dev(64, dtype=F32), cu(6000), None, x, **kw).values()


def b_qk_norm(**kw):
    return mm.qk_norm(dev(6, 4, 64), dev(6, 2, 64), dev(64, dtype=F32), dev(64, dtype=F32), **kw)


def b_qk_norm_backward(**kw):
    q, k, w = dev(6, 4, 64), dev(6, 2, 64), dev(64, dtype=F32)
    return mm.qk_norm_backward(q, k, q, k, w, w, **kw)


BOUND = [b_conv_prefill, b_conv_decode, b_conv_backward, b_gated_prefill, b_gated_prefill_train, b_gated_decode, b_gated_backward,
         b_qk_norm, b_qk_norm_backward]


@pytest.mark.parametrize("call", BOUND, ids=[c.__name__[2:] for c in BOUND])
def test_allocations_belong_to_the_given_stream(call):
    outputs = [t for t in call(stream=SIDE) if t is not None]
    log = streams.LOG
    assert len(log.launched) == 1 and SIDE.cuda_stream in log.launched[0]
    assert log.made and all(stream is SIDE for _, stream in log.made)
    used = {p for p, stream in log.used if stream is CURRENT}
    assert used == {t.data_ptr() for t in outputs}, "the current stream will use the outputs, and they alone"


@pytest.mark.parametrize("call", BOUND, ids=[c.__name__[2:] for c in BOUND])
def test_allocations_of_a_call_on_the_current_stream(call, monkeypatch):
    import selective_state_space_causal_amd.heads as binding

    monkeypatch.setattr(binding, "_raw_stream", lambda index: CURRENT.cuda_stream)
    call()
    log = streams.LOG
    assert log.made and all(stream is None for _, stream in log.made) and not log.used


# ---------------------------------------------------------------------------- references against differences
def slope_of(loss, c, k, v, e=1e-5):
    return (loss(dict(c, **{k: c[k].double() + e * v})) - loss(dict(c, **{k: c[k].double() - e * v}))) / (2 * e)


def direction(t, seed=3):
    return torch.randn(t.shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradients_against_differences(silu):
    c = ref.conv_inputs(5, [9, 0, 2, 20], 5, 4, "f32")
    want = ref.conv_backward(c, silu)

    def loss(k):
        y, s, _ = ref.conv(k, silu)
        return float((y * c["dy"].double()).sum() + (s * c["dstate"].double()).sum())

    for k, n in dict(x="dx", weight="dweight", bias="dbias", state="dstate_in").items():
        v = direction(c[k])
        mine = float((want[n][0] * v).sum())
        assert abs(mine - slope_of(loss, c, k, v)) <= 1e-6 * (1 + abs(mine)), k


@pytest.mark.parametrize("lam,g,z,gate", [(True, True, True, "gelu"), (False, False, True, "silu"), (True, False, False, "silu")])
def test_gated_gradients_against_differences(lam, g, z, gate):
    c = ref.gated_inputs(6, [9, 0, 20], 5, "f32", lam, g, z)
    want = ref.gated_backward(c, gate)

    def loss(k):
        y, s = ref.gated(k, gate)[:2]
        return float((y * c["dy"].double()).sum() + (s * c["dstate"].double()).sum())

    for k, n in dict(x="dx", r="dr", g="dg", z="dz", lam="dlam", state="dstate_in").items():
        if c[k] is None:
            assert n not in want
            continue
        v = direction(c[k])
        mine = float((want[n][0] * v).sum())
        assert abs(mine - slope_of(loss, c, k, v)) <= 1e-6 * (1 + abs(mine)), k


@pytest.mark.parametrize("inter", [True, False])
def test_qk_gradients_against_differences(inter):
    c = ref.qk_inputs(7, 6, 3, 2, 10, 6, "f32", far=50)
    want = ref.qk_backward(c, inter)

    def loss(k):
        (q, _), (kk, _) = ref.qk(k, inter)
        return float((q * c["dq"].double()).sum() + (kk * c["dk"].double()).sum())

    for k, n in dict(q="dq", k="dk", wq="dwq", wk="dwk").items():
        v = direction(c[k])
        mine = float((want[n][0] * v).sum())
        assert abs(mine - slope_of(loss, c, k, v)) <= 1e-6 * (1 + abs(mine)), k
