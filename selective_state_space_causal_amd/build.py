"""Build libmambamix.so in-tree with hipcc for gfx950."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SRC = [os.path.join(CSRC, f) for f in ("mambamix.hip", "heads.hip", "layer/conv.hip", "layer/gated.hip", "layer/qk_norm.hip")]
LIB = os.path.join(HERE, "libmambamix.so")
INCLUDE = os.path.join(ROOT, "include")

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-shared", "--offload-arch=gfx950",
    # keep the compiler from forming packed fp32 (v_pk_*_f32) instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(verbose: bool = False) -> str:
    """Compile the HIP library (always recompiles) and return its path."""
    objs, running = [], []
    for src in SRC:
        objs.append(f"{LIB}.{os.path.basename(src)}.o")
        cmd = [hipcc(), *[f for f in HIPCC_FLAGS if f != "-shared"], "-I", INCLUDE, "-I", CSRC, "-c", "-o", objs[-1], src]
        running.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    said = "".join(p.communicate()[0] for p in running)
    tmp = LIB + ".tmp"
    if all(p.returncode == 0 for p in running):
        res = subprocess.run([hipcc(), "-shared", "-fPIC", "--offload-arch=gfx950", "-o", tmp, *objs],
                             capture_output=True, text=True)
        said += res.stdout + res.stderr
        ok = res.returncode == 0
    else:
        ok = False
    for o in objs:
        if os.path.exists(o):
            os.remove(o)
    if not ok:
        sys.stderr.write(said)
        raise RuntimeError("hipcc failed to build libmambamix")
    if verbose:
        sys.stderr.write(said)
    os.replace(tmp, LIB)
    return LIB


def asm(out: str) -> None:
    """Write the gfx950 device assembly of the library to ``out`` (for inspection), one source after another."""
    text = ""
    for src in SRC:
        cmd = [hipcc(), *[f for f in HIPCC_FLAGS if f not in ("-shared", "-fPIC")], "-I", INCLUDE, "-I", CSRC,
               "--cuda-device-only", "-S", "-o", out, src]
        subprocess.run(cmd, check=True, capture_output=True)
        with open(out) as f:
            text += f.read()
    with open(out, "w") as f:
        f.write(text)


if __name__ == "__main__":
    print(build(verbose=True))
