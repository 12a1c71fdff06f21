"""The units of the convolution, the gated recurrence and the head norm: their sources are all found, a change makes the rocprofv3
summaries of its own unit stale and no others, and each kernel has one."""
from __future__ import annotations

import os
import shutil

import pytest

import bench
from selective_state_space_causal_amd import build

UNITS = sorted(os.path.relpath(s, build.CSRC) for s in build.SRC)
LAYER = [u for u in UNITS if u.startswith("layer/")]
SUMMARIES = {"layer/conv.hip": ("k_conv__", "k_conv_bwd__"), "layer/gated.hip": ("k_gated__", "k_gated_bwd__"),
             "layer/qk_norm.hip": ("k_qk_rows__", "k_qk_rows_bwd__")}


def test_every_source_is_of_a_unit():
    assert LAYER == sorted(SUMMARIES)
    every = {os.path.relpath(os.path.join(at, f), build.CSRC) for at, _, files in os.walk(build.CSRC) for f in files
             if f.endswith((".hip", ".h"))}
    assert set().union(*(bench.kernel_sources(u) for u in UNITS)) == every


@pytest.mark.parametrize("changed", ["layer/common.h", "layer/conv.hip", "layer/gated.hip", "layer/qk_norm.hip", "mm_device.h", "mm_norm.h"])
def test_a_change_makes_the_summaries_of_its_own_units_stale(tmp_path, changed):
    folder = str(tmp_path / "csrc")
    shutil.copytree(build.CSRC, folder)
    before = [bench.kernel_source_sha256(u, folder) for u in LAYER]
    assert before == [bench.kernel_source_sha256(u) for u in LAYER]
    with open(os.path.join(folder, changed), "a") as f:
        f.write("\n// changed\n")
    after = [bench.kernel_source_sha256(u, folder) for u in LAYER]
    hit = {"layer/common.h": LAYER, "mm_device.h": LAYER, "mm_norm.h": []}.get(changed, [changed])
    assert [u for u, a, b in zip(LAYER, after, before) if a != b] == hit


@pytest.mark.parametrize("unit", SUMMARIES)
def test_each_kernel_has_a_summary(unit):
    found = os.listdir(os.path.join(bench.ROOT, "profiles"))
    for kernel in SUMMARIES[unit]:
        assert sum(f.startswith(kernel) for f in found) == 1, kernel
