"""The instances that large calls take, at sizes a test can afford: whole sequences of several chunks in the prefill
and both sides of its choice, state walks that are not sliced, and gradient workgroups that take several heads.  Which
instance a case takes follows from the library's rules, repeated here, so that a case that stops reaching its
instance fails.  Needs an MI355X."""
from __future__ import annotations

import math

import pytest
import torch

import selective_state_space_causal_amd as mm
from tests import heads_ref as ref
from tests.test_gpu_heads import check_backward, check_prefill, run_backward, run_prefill, to_gpu, tokens

pytestmark = pytest.mark.gpu

CUS, TOK = 256, 64


def cdiv(a, b):
    return -(-a // b)


def prefill_stretch(lens, H, P, G):
    """(stretch length, whether whole sequences run) of a bfloat16 prefill with N <= 128."""
    S, T = len(lens), sum(lens)
    pairs = G * cdiv(H // G * cdiv(P, 64), 2)
    enough = S * pairs >= 2 * CUS
    least = int(math.sqrt(0.5 * T * pairs))
    Ls = max(1, cdiv(max(least, cdiv(T, max(1, 2 * CUS // pairs))), TOK)) * TOK
    if (enough and S > 256) or Ls >= T:
        return Ls, True
    return Ls, enough and max(lens) <= 2 * Ls


# lens, H, P, G, N; whole sequences?; the last column: chunks of the longest sequence
PREFILL = {
    "at two stretches of 64": ([3] * 63 + [128], 16, 64, 8, 100, True, 2),
    "past two stretches of 64": ([3] * 63 + [129], 16, 64, 8, 100, False, 3),
    "at two stretches of 128": ([13] * 63 + [256], 16, 64, 8, 32, True, 4),
    "past two stretches of 128": ([13] * 63 + [257], 16, 64, 8, 32, False, 5),
    "odd lengths": ([65, 127, 200, 0, 1, 64] * 11, 16, 64, 8, 128, True, 4),
    "odd lengths, half a pair": ([65, 127, 200] * 29, 6, 80, 2, 50, True, 4),
    "more than 256 sequences": ([2] * 300 + [70, 0, 150], 4, 64, 2, 64, True, 3),
    "one head of 20 channels": ([66, 3] * 260, 1, 20, 1, 24, True, 2),
}


@pytest.mark.parametrize("name", PREFILL)
def test_prefill_of_whole_sequences(name):
    lens, H, P, G, N, whole, chunks = PREFILL[name]
    assert prefill_stretch(lens, H, P, G)[1] == whole and cdiv(max(lens), TOK) == chunks
    c = ref.heads_inputs(31, lens, H, P, G, N, "bf16")
    check_prefill(c, *run_prefill(c))


@pytest.mark.parametrize("shape", [(16, 64, 8, 128), (16, 64, 8, 100)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_values_that_are_not_finite_in_whole_sequences(shape, value):
    """They reach their own sequence only, from their token on, also in the chunks after it."""
    H, P, G, N = shape
    lens = [65, 200, 70] * 22
    assert prefill_stretch(lens, H, P, G)[1]
    c = ref.heads_inputs(32, lens, H, P, G, N, "bf16")
    clean_y, clean_s = run_prefill(c)
    at, lo, hi = 65 + 100, 65, 265
    for key in ("x", "B"):
        d = dict(c, proj=c["proj"].clone())
        ref.split(d)
        d[key][at] = value
        y, s = run_prefill(d)
        assert torch.equal(y[:lo], clean_y[:lo]) and torch.equal(y[hi:], clean_y[hi:]), f"{key}: other sequences"
        assert torch.isfinite(y[lo:at]).all(), f"{key}: earlier tokens"
        assert (y[lo:at].float() - clean_y[lo:at].float()).abs().max() <= 0.05 * clean_y.float().abs().max()
        assert torch.equal(s[0], clean_s[0]) and torch.equal(s[2:], clean_s[2:])
        assert not torch.isfinite(y[at]).all() and not torch.isfinite(y[at + 64:hi]).any() and not torch.isfinite(s[1]).any()


@pytest.mark.parametrize("N", [128, 100])
def test_prefill_state_walks_of_all_columns(N):
    lens, H, P, G = [1100, 0, 300, 600], 64, 16, 1
    Ls, whole = prefill_stretch(lens, H, P, G)
    assert not whole and cdiv(sum(lens), Ls) * H * cdiv(P, 64) > 2 * CUS
    c = ref.heads_inputs(33, lens, H, P, G, N, "bf16")
    check_prefill(c, *run_prefill(c))


@pytest.mark.parametrize("N", [128, 100])
def test_backward_state_walks_of_all_columns(N):
    lens, H, P, G = [70, 130, 0, 1, 64, 65, 33, 2, 90], 30, 16, 2
    assert len(lens) * H * cdiv(P, 64) * 2 > 2 * CUS
    c = ref.heads_inputs(34, lens, H, P, G, N, "bf16")
    check_backward(c, run_backward(c))


def head_shares(lens, H, G):
    """How many workgroups of the gradient kernel share the heads of a (block, group)."""
    return max(1, min(H // G, cdiv(2 * CUS, (len(lens) + sum(lens) // TOK) * G)))


@pytest.mark.parametrize("H,P,G,N", [(7, 64, 1, 128), (7, 80, 1, 50), (7, 20, 1, 16), (10, 64, 2, 100), (5, 130, 1, 32)])
def test_backward_of_several_heads_a_workgroup(H, P, G, N):
    lens = [3] * 150 + [70, 0, 129]
    shares, heads = head_shares(lens, H, G), H // G
    assert shares < heads and heads % shares != 0, "unequal shares, of more than one head"
    c = ref.heads_inputs(35, lens, H, P, G, N, "bf16")
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("no", ["dt", "D"])
def test_backward_of_several_heads_a_workgroup_without(no):
    lens, H, P, G, N = [3] * 150 + [70], 7, 64, 1, 64
    assert head_shares(lens, H, G) < H
    c = ref.heads_inputs(36, lens, H, P, G, N, "bf16", no != "dt", no != "D")
    check_backward(c, run_backward(c))


@pytest.mark.parametrize("lens", [[40, 3], [300]])
def test_rows_too_far_apart_for_the_matrix_cores(lens):
    """x in rows of more than 2^22 elements: token by token, in the workspace that the binding asks for then."""
    T, far = sum(lens), 4194304 + 8
    c = ref.heads_inputs(37, lens, 2, 16, 1, 32, "bf16")
    g = to_gpu(c)
    wide = torch.empty(T * far, dtype=torch.bfloat16, device="cuda").as_strided((T, 2, 16), (far, 16, 1))
    wide.copy_(g["x"])
    args = [wide] + tokens(g)[1:]
    y, s = mm.heads_prefill(*args, g["cu"], g["state"])
    check_prefill(c, y, s)
    check_backward(c, mm.heads_backward(*args, g["cu"], g["state"], g["dy"], g["dstate"]))
