"""Build the gfx950 shared library ``libtopselect.so`` in-tree with hipcc.

Usage: ``python -m top_select_gumbel_amd.build`` (or ``build()`` from Python).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", f) for f in ("topselect.hip", "rejection.hip", "read_ceiling.hip", "logprobs.hip",
                                               "evict.hip")]
INC = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtopselect.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # packed fp32 VALU forms stay off (see the design notes)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fno-gpu-flush-denormals-to-zero",
    "-Wno-unused-result",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain (ROCm) is required to build libtopselect.so")


def build(verbose: bool = False) -> str:
    """Compile libtopselect.so (always recompiles, a process a source). Returns the library path."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as work:
        objs = [os.path.join(work, os.path.basename(src) + ".o") for src in SRCS]
        jobs = []
        for src, obj in zip(SRCS, objs):
            cmd = [hipcc(), *HIPCC_FLAGS, "-I", INC, "-I", os.path.join(PKG, "csrc"), "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
        outs = [job.communicate()[0] for job in jobs]
        for job, out in zip(jobs, outs):
            if job.returncode != 0:
                raise RuntimeError("hipcc failed:\n" + out[-12000:])
        res = subprocess.run([hipcc(), "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", tmp], capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("linking failed:\n" + res.stdout[-4000:] + res.stderr[-8000:])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
