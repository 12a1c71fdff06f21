"""The norms with more rows than workgroups: the loop over rows, the next row's loads under this one's sums, and the
weights' gradients gathered over the rows of a workgroup.  How many rows run at once follows from the library's rule,
repeated here.  Needs an MI355X."""
from __future__ import annotations

import pytest

from tests import test_gpu_norms as norms

pytestmark = pytest.mark.gpu

WAVE, CUS, MOST = 64, 256, 1024


def cdiv(a, b):
    return -(-a // b)


def slots(n, groups, backward):
    """Rows (of one group) that run at once, n columns each."""
    pieces = cdiv(n, 4)
    t = cdiv(cdiv(pieces, 2 if pieces > MOST else 1), WAVE) * WAVE
    return cdiv(CUS * (max(1, 24 * WAVE // t) if backward else max(16, 8192 // t)), groups)


# rows, d, groups, io
GATE = [(1100, 64, 64, "bf16"), (1100, 320, 64, "f32"), (4200, 1801, 1, "bf16"), (4100, 2056, 1, "bf16")]
GATE_BACKWARD = [(1100, 64, 64, "bf16"), (700, 320, 64, "f32"), (600, 2049, 1, "bf16"), (1100, 5120, 8, "bf16"),
                 (700, 2560, 1, "f32"), (300, 8000, 1, "f32"), (301, 8192, 1, "bf16")]


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("rows,d,groups,io", GATE)
def test_gate_norm(rows, d, groups, io, gate_first):
    assert rows > slots(d // groups, groups, False)
    norms.test_gate_norm(rows, d, groups, io, gate_first)


@pytest.mark.parametrize("gate_first", [True, False])
@pytest.mark.parametrize("rows,d,groups,io", GATE_BACKWARD)
def test_gate_norm_backward(rows, d, groups, io, gate_first):
    assert rows > slots(d // groups, groups, True)
    norms.test_gate_norm_backward(rows, d, groups, io, gate_first)


@pytest.mark.parametrize("post,vec", [(True, True), (False, False)])
@pytest.mark.parametrize("rows,d,io,res", [(4200, 1801, "bf16", "f32"), (4100, 2056, "bf16", "bf16")])
def test_residual_norm(rows, d, io, res, post, vec):
    assert rows > slots(d, 1, False)
    norms.test_residual_norm(rows, d, io, res, post, vec)


@pytest.mark.parametrize("post,vec", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows,d,io,res", [(600, 2560, "bf16", "f32"), (600, 4096, "bf16", "bf16"), (300, 8000, "f32", "f32"),
                                           (700, 2049, "bf16", "f32"), (301, 8192, "bf16", "bf16")])
def test_residual_norm_backward(rows, d, io, res, post, vec):
    assert rows > slots(d, 1, True)
    norms.test_residual_norm_backward(rows, d, io, res, post, vec)
