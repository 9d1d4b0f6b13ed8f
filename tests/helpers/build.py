"""Builds the GPU test helpers in tests/helpers/ (hipcc, gfx950) into
tests/helpers/_build/: the programs, and libforced_plan.so and
libforced_moe_plan.so, the gradient operators and the experts' with tile and
split chosen by the test (plans/).
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
    csrc, plans = zbuild.CSRC, os.path.join(HERE, "plans")
    # each with the library's sources that its operators need
    libs = {"forced_plan": ("train_api", "train_rows"),
            "forced_moe_plan": ("moe_api", "moe_back_gemm", "moe_depth_gemm", "moe_route", "moe_rows")}
    for name, rest in libs.items():
        lib = os.path.join(OUT, f"lib{name}.so")
        zbuild.compile_and_link([os.path.join(plans, name + ".hip"),
                                 *(os.path.join(csrc, r + ".hip") for r in rest)], lib)
        built.append(lib)
    return built


if __name__ == "__main__":
    print("\n".join(build()))
