"""Builds the GPU test helpers in tests/helpers/ (hipcc, gfx950) into
tests/helpers/_build/: the programs, and libforced_plan.so, the gradient
operators with tile and split chosen by the test (plans/forced_plan.hip).
Called by __graft_entry__.build(); runs without a GPU."""
from __future__ import annotations

import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from sharded_optimizer_step_adamw_amd import build as zbuild  # noqa: E402

OUT = os.path.join(HERE, "_build")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def build() -> list:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    os.makedirs(OUT, exist_ok=True)
    built = []
    for src in sorted(glob.glob(os.path.join(HERE, "*.hip"))):
        exe = os.path.join(OUT, os.path.splitext(os.path.basename(src))[0])
        subprocess.run([hipcc, *FLAGS, src, "-o", exe + ".tmp"], check=True)
        os.replace(exe + ".tmp", exe)
        built.append(exe)
    lib = os.path.join(OUT, "libforced_plan.so")
    csrc = zbuild.CSRC
    subprocess.run([hipcc, *zbuild.HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-I", csrc,
                    os.path.join(HERE, "plans", "forced_plan.hip"), os.path.join(csrc, "train_api.hip"),
                    os.path.join(csrc, "train_rows.hip"), "-o", lib + ".tmp"], check=True)
    os.replace(lib + ".tmp", lib)
    return built + [lib]


if __name__ == "__main__":
    print("\n".join(build()))
