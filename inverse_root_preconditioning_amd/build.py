"""Build the HIP library in-tree: lib/libshampoo_mi355x.so for gfx950.

    python -m inverse_root_preconditioning_amd.build

hipcc cross-compiles without a GPU.  Packed fp32 instructions are disabled
for all device code (`-packed-fp32-ops`); the host pass warns that it does
not know that feature, which is harmless.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libshampoo_mi355x.so")
ARCH = os.environ.get("SHAMPOO_OFFLOAD_ARCH", "gfx950")

SOURCES = ["shampoo.hip", "adamw.hip", "mx4.hip"]
HEADERS = ["common.h", "gemm_f32.h", "gemm_bf16.h", "kernels_misc.h", "vector_io.h", "kernels_adamw.h", "kernels_mx4.h"]


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def compile_command(source, out):
    return [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"),
            "-o", out, os.path.join(CSRC, source)]


def link_command(objects, out):
    return [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", out] + objects


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build(verbose=False):
    """Compile the library (always recompiles, its sources side by side).  Raises on failure."""
    os.makedirs(LIBDIR, exist_ok=True)
    objects = [os.path.join(LIBDIR, s + ".o") for s in SOURCES]
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        list(ex.map(lambda job: _run(compile_command(*job), verbose), zip(SOURCES, objects)))
    tmp = LIB + ".tmp"
    _run(link_command(objects, tmp), verbose)
    for o in objects:
        os.remove(o)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
