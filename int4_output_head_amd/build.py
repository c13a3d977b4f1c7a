"""Build step of the package: compiles the HIP library for gfx950 in-tree."""
from __future__ import annotations

import ctypes
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = ("int4vh.hip", "requant.hip", "context_copy.hip", "stream_probe.hip", "norm.hip", "linear.hip",
           "logits.hip", "mxfp4.hip", "sample.hip")
SRCS = [os.path.join(HERE, "csrc", f) for f in SOURCES]
OUT = os.path.join(HERE, "libint4vh.so")
INCLUDE = os.path.join(ROOT, "include")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # no packed-fp32 instructions in generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def build_library(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = OUT + ".tmp"

    def run(args):
        cmd = [hipcc, *HIPCC_FLAGS, *args]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed ({r.returncode}):\n{r.stdout}\n{r.stderr}")

    # the sources side by side: one after another they take minutes
    with tempfile.TemporaryDirectory() as objects, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        built = [os.path.join(objects, f + ".o") for f in SOURCES]
        list(pool.map(lambda s, o: run(["-c", "-I", INCLUDE, s, "-o", o]), SRCS, built))
        run(["-shared", *built, "-o", tmp])
    # hipcc can finish without an error yet leave a kernel's host stub
    # undefined; such a library fails at load time, so check that here.
    try:
        ctypes.CDLL(tmp, mode=os.RTLD_NOW)
    except OSError as e:
        os.unlink(tmp)
        raise RuntimeError(f"built library does not load: {e}") from None
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build_library(verbose=True))
