"""Build libzopt.so in-tree for gfx950 with hipcc.

    python -m sharded_optimizer_step_adamw_amd.build

All kernel sources and the C-ABI entry points are compiled, side by side, and
linked into one shared library next to this file.  Packed-fp32 instructions
are disabled (the compiler would otherwise pair fp32 operations into them).
Only the entry points declared in include/zopt.h are exported.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libzopt.so")
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-shared", "-fPIC",
    "-fvisibility=hidden", "-Wall", "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def compile_and_link(files, out: str, verbose: bool = False) -> str:
    """One object a source, at most 8 at a time, linked into `out`."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as tmp:

        def compile_one(src):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            cmd = [hipcc, *flags, "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
            return obj

        with concurrent.futures.ThreadPoolExecutor(8) as pool:
            objects = list(pool.map(compile_one, files))
        # (whoever has the library loaded keeps the file that it loaded)
        subprocess.run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objects, "-o", out + ".tmp"], check=True)
    os.replace(out + ".tmp", out)
    return out


def build(verbose: bool = False) -> str:
    return compile_and_link(sources(), LIB, verbose)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
