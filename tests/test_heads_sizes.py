"""Sizes at the launches' limits, on the host with device addresses that are never touched: what a call can run is not
refused for a limit of another one's."""
from __future__ import annotations

import ctypes

from tests.test_heads_host import ALIAS, DIM, WORKSPACE, backward, gate, gate_backward, lib, prefill  # noqa: F401

FAR = 1 << 40  # no two arrays overlap


def far(n):
    return [ctypes.c_void_p((i + 1) * FAR) for i in range(n)]


def sizes(T, H=64, P=64, G=1, N=128, io=1):
    return dict(S=3, T=T, H=H, P=P, G=G, N=N, io=io, xs=H * P, ds=H, bs=G * N, cs=G * N, ws=0, wsb=0)


def grads(T, **kw):
    c = sizes(T, **kw)
    return dict(c, gx=c["xs"], gd=c["ds"], gb=c["bs"], gc=c["cs"])


def test_a_prefill_has_no_limit_of_tokens_times_heads(lib):  # noqa: F811
    for T in ((1 << 28) // 64 + 1, 5_000_000, 16_000_000):
        assert prefill(lib, far(11), **sizes(T)) == WORKSPACE, T
        assert lib.mamba_mixer_heads_prefill_workspace_bytes(3, T, 64, 64, 1, 128, 1) > 0, T
    assert prefill(lib, far(11), **sizes(5_000_000, io=0)) == WORKSPACE
    assert prefill(lib, far(11), **sizes(5_000_000, N=256)) == WORKSPACE


def test_a_backward_on_the_matrix_cores_has_none_either(lib):  # noqa: F811
    for T in ((1 << 28) // 64 + 1, 5_000_000):
        assert backward(lib, far(19), **grads(T, N=16)) == WORKSPACE, T
        assert lib.mamba_mixer_heads_backward_workspace_bytes(3, T, 64, 64, 1, 16, 1) > 0, T
    assert backward(lib, far(19), **grads(5_000_000, G=8, N=128)) == DIM  # T G N: the gradients of B and C


def test_the_float32_backward_has(lib):  # noqa: F811
    """A workgroup for each (64-token block, head)."""
    fits = 64 * ((1 << 18) - 3) - 1
    assert backward(lib, far(19), **grads(fits, N=16, io=0)) == WORKSPACE
    assert lib.mamba_mixer_heads_backward_workspace_bytes(3, fits, 64, 64, 1, 16, 0) > 0
    assert backward(lib, far(19), **grads(fits + 65, N=16, io=0)) == DIM


def test_gate_norm_of_more_groups_than_a_launch_has_workgroups(lib):  # noqa: F811
    """Refused on the host as sizes, not by the launch."""
    d = 1 << 26
    wide = dict(rows=2, d=d, ys=d, zs=d)
    assert gate(lib, far(4), g=d, **wide) == DIM
    p = far(4)
    p[3] = p[1]
    assert gate(lib, p, g=d // 2, **wide) == ALIAS  # half as many are accepted: past the sizes
    grads = dict(wide, gy=d, gz=d, wsb=0)
    assert gate_backward(lib, far(7), g=d, **grads) == DIM
    assert gate_backward(lib, far(7), g=d // 2, **grads) == WORKSPACE
    d = 1 << 28  # the weights' sums: 16 threads a column
    assert gate_backward(lib, far(7), rows=2, d=d, g=8, ys=d, zs=d, gy=d, gz=d, wsb=0) == DIM
    assert lib.mamba_mixer_gate_norm_backward_workspace_bytes(2, d, 8) == 0
