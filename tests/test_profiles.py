"""The committed rocprofv3 summaries are tied to the sources of the kernel they describe, and to those alone."""
from __future__ import annotations

import glob
import os
import re
import shutil

import pytest

import bench

PROFILES = sorted(glob.glob(os.path.join(bench.ROOT, "profiles", "*.txt")))


def test_the_units_sources():
    scan, heads = bench.kernel_sources("mambamix.hip"), bench.kernel_sources("heads.hip")
    assert {"mambamix.hip", "mm_row.h", "mm_device.h"} <= set(scan) and not {"heads.hip", "mm_heads.h", "mm_norm.h"} & set(scan)
    assert {"heads.hip", "mm_heads_mma.h", "mm_norm.h", "mm_device.h"} <= set(heads) and "mm_row.h" not in heads
    every = {f for f in os.listdir(bench.KERNEL_DIR) if f.endswith((".hip", ".h"))}
    assert set(scan) | set(heads) == every, "a source of no unit"


@pytest.mark.parametrize("changed", ["heads.hip", "mm_heads_grad.h", "mm_norm.h", "mm_row.h", "mm_device.h"])
def test_a_change_makes_the_summaries_of_its_own_units_stale(tmp_path, changed):
    folder = str(tmp_path / "csrc")
    shutil.copytree(bench.KERNEL_DIR, folder)
    units = ("mambamix.hip", "heads.hip")
    before = [bench.kernel_source_sha256(u, folder) for u in units]
    assert before == [bench.kernel_source_sha256(u) for u in units]
    with open(os.path.join(folder, changed), "a") as f:
        f.write("\n// changed\n")
    after = [bench.kernel_source_sha256(u, folder) for u in units]
    assert [a != b for a, b in zip(after, before)] == [changed in bench.kernel_sources(u, folder) for u in units]


@pytest.mark.parametrize("path", PROFILES, ids=[os.path.basename(p) for p in PROFILES])
def test_every_summary_names_its_sources(path):
    text = open(path).read()
    assert len(re.findall(r"^kernel source sha256: [0-9a-f]{64}$", text, re.M)) == 1
