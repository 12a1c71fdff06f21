"""Lanes of a wave that exchange values through LDS: the program itself orders the accesses.  A wave barrier alone is no memory
operation to the compiler, which may then move one lane's load over another's store; each has to stand between a release and
an acquire.  Read from the device IR that the compiler starts from, without a GPU."""
from __future__ import annotations

import os
import subprocess

import pytest

from selective_state_space_causal_amd import build

UNITS = [os.path.relpath(s, build.CSRC) for s in build.SRC]


@pytest.mark.parametrize("unit", UNITS)
def test_wave_barriers_stand_between_fences(unit, tmp_path):
    if not os.path.exists(build.hipcc()):
        pytest.skip("hipcc not installed")
    out = tmp_path / "unit.ll"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([build.hipcc(), *flags, "-I", build.INCLUDE, "-I", build.CSRC, "--cuda-device-only", "-S", "-emit-llvm", "-Xclang",
                    "-disable-llvm-passes", "-o", str(out), os.path.join(build.CSRC, unit)], check=True, capture_output=True)
    lines = [line.strip() for line in out.read_text().splitlines()]
    at = [i for i, line in enumerate(lines) if line.startswith("call void @llvm.amdgcn.wave.barrier()")]
    for i in at:
        before, after = lines[i - 1], lines[i + 1]
        # an acquire-release fence ahead of it orders both sides: the barrier itself is no access
        assert before.startswith("fence ") and ("acq_rel" in before or "release" in before and after.startswith("fence ")
                                                and "acquire" in after), "\n".join(lines[i - 3:i + 4])
    if unit == "layer/qk_norm.hip":
        assert at, "the rows of any width exchange through LDS"
