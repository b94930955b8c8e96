"""Compile the HIP library libpdgemm.so for gfx950, in place."""
from __future__ import annotations

import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", name) for name in ("pdgemm.hip", "mxfp4.hip", "rmsnorm.hip", "a16_i4.hip", "moe.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(HERE, "libpdgemm.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # no packed-fp32 VALU instructions in any generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIBRARY + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        # (the sources side by side: each takes minutes)
        jobs, outputs = [], []
        for source in SOURCES:
            outputs.append(os.path.join(objects, os.path.basename(source) + ".o"))
            cmd = [hipcc, *HIPCC_FLAGS, "-I", INCLUDE, "-c", source, "-o", outputs[-1]]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append((cmd, subprocess.Popen(cmd)))
        failed = [cmd for cmd, job in jobs if job.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        subprocess.check_call([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", *outputs, "-o", tmp])
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose=True))
