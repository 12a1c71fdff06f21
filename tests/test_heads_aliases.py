"""In place means one output over one input: an output at the address of an input is refused unless that pair is the
documented one, whatever else shares the address.  On the host, with device addresses that are never touched."""
from __future__ import annotations

import pytest

from tests.test_heads_host import (ALIAS, WORKSPACE, at, backward, decode, gate, gate_backward, lib, prefill,  # noqa: F401
                                   ptrs, residual, residual_backward)

# call, its arguments, the outputs' places, the inputs' places, the pairs (output, input) that may be one
CALLS = [
    (prefill, 11, (9, 10), tuple(range(9)), {(9, 8)}, dict(wsb=0)),
    (decode, 10, (8, 9), tuple(range(8)), {(8, 7)}, dict()),
    (backward, 19, tuple(range(11, 19)), tuple(range(11)), set(), dict(wsb=0)),
    (gate, 4, (3,), (0, 1, 2), {(3, 0)}, dict()),
    (gate_backward, 7, (4, 5, 6), (0, 1, 2, 3), set(), dict(wsb=0)),
    (residual, 7, (5, 6), (0, 1, 2, 3, 4), {(5, 1)}, dict()),
    (residual_backward, 12, tuple(range(7, 12)), tuple(range(7)), {(7, 1)}, dict(wsb=0)),
]


@pytest.mark.parametrize("call,n,outs,ins,same,kw", CALLS, ids=[c[0].__name__ for c in CALLS])
def test_only_the_documented_pairs_may_be_one(lib, call, n, outs, ins, same, kw):  # noqa: F811
    p = ptrs(n)
    for o in outs:
        for i in ins:
            if (o, i) not in same:
                assert call(lib, at(p, o, p[i].value), **kw) == ALIAS, (o, i)


@pytest.mark.parametrize("call,n,outs,ins,same,kw", [c for c in CALLS if c[4]], ids=[c[0].__name__ for c in CALLS if c[4]])
def test_another_array_at_the_in_place_address(lib, call, n, outs, ins, same, kw):  # noqa: F811
    """A second input, or a second output, where an output is written over its input."""
    p = ptrs(n)
    (o, i), = same
    q = at(p, o, p[i].value)
    for k in (*ins, *outs):
        if k not in (o, i):
            assert call(lib, at(q, k, p[i].value), **kw) == ALIAS, k


def test_the_documented_pairs_are_accepted(lib):  # noqa: F811
    """Past the overlap checks: the next refusal is the workspace's."""
    for call, n, _, _, same, kw in CALLS:
        if same and kw:
            (o, i), = same
            p = ptrs(n)
            assert call(lib, at(p, o, p[i].value), **kw) == WORKSPACE, call.__name__
