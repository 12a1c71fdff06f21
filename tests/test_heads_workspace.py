"""The workspace that the queries ask for is the one that a call uses, not the larger one of a path that it does not take.
On the host, with device addresses that are never touched."""
from __future__ import annotations

import pytest

import selective_state_space_causal_amd.heads as binding
from tests.test_heads_host import ALIGN, WORKSPACE, backward, lib, prefill  # noqa: F401
from tests.test_heads_sizes import far, grads, sizes

WIDE = 4194304 + 8  # elements between rows: past the matrix-core kernels


def cases(lib, call):  # noqa: F811
    name, n, make = ("prefill", 11, sizes) if call is prefill else ("backward", 19, grads)
    query = getattr(lib, f"mamba_mixer_heads_{name}_workspace_bytes")
    return n, make, lambda io, T, N: query(3, T, 64, 64, 1, N, io)


@pytest.mark.parametrize("call", [prefill, backward])
@pytest.mark.parametrize("io,N", [(1, 128), (1, 200), (0, 64)])
def test_the_query_is_what_the_call_needs(lib, call, io, N):  # noqa: F811
    n, make, query = cases(lib, call)
    for T in (700, 20000):
        need = query(io, T, N)
        kw = make(T, N=N, io=io)
        assert need > 0
        assert call(lib, far(n), **dict(kw, ws=0x7F00000010, wsb=need)) == ALIGN, "enough: the next check refuses"
        assert call(lib, far(n), **dict(kw, ws=0x7F00000000, wsb=need - 1)) == WORKSPACE


@pytest.mark.parametrize("call", [prefill, backward])
def test_wider_rows_need_the_float32_one(lib, call):  # noqa: F811
    n, make, query = cases(lib, call)
    for row in ("xs", "bs", "cs"):
        kw = dict(make(20000, N=128), **{row: WIDE})
        assert call(lib, far(n), **dict(kw, ws=0x7F00000010, wsb=query(0, 20000, 128))) == ALIGN
        assert call(lib, far(n), **dict(kw, ws=0x7F00000000, wsb=query(0, 20000, 128) - 1)) == WORKSPACE
    assert binding._plan_code(1, 256, 4, 256, 4194304) == 1 and binding._plan_code(1, 256, 4, WIDE) == 0


def test_a_training_step_does_not_ask_for_the_token_by_token_states(lib):  # noqa: F811
    query = lib.mamba_mixer_heads_backward_workspace_bytes
    assert query(8, 16384, 24, 64, 1, 128, 1) < 0.6 * query(8, 16384, 24, 64, 1, 128, 0)
