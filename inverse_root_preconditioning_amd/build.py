"""Build in-tree the HIP library, lib/libshampoo_mi355x.so for gfx950, and the
torch extension over it, lib/_layers.so (host code only).

    python -m inverse_root_preconditioning_amd.build

hipcc cross-compiles without a GPU.  Packed fp32 instructions are disabled
for all device code (`-packed-fp32-ops`); the host pass warns that it does
not know that feature, which is harmless.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libshampoo_mi355x.so")
LAYERS = os.path.join(LIBDIR, "_layers.so")
ARCH = os.environ.get("SHAMPOO_OFFLOAD_ARCH", "gfx950")

SOURCES = ["shampoo.hip", "adamw.hip", "mx4.hip", "layers.hip", "norm.hip", "norm_back_bf16.hip", "norm_back_f32.hip",
           "norm_back_mixed.hip"]
HEADERS = ["common.h", "gemm_f32.h", "gemm_bf16.h", "kernels_misc.h", "vector_io.h", "kernels_adamw.h", "kernels_mx4.h",
           "host.h", "kernels_mx8.h", "kernels_act.h", "kernels_norm.h", "kernels_norm_sums.h", "norm_launch.h"]


def rocm():
    return os.environ.get("ROCM_PATH", "/opt/rocm")


def hipcc():
    return os.path.join(rocm(), "bin", "hipcc")


def compile_command(source, out):
    return [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-c",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-I", os.path.join(ROOT, "include"),
            "-o", out, os.path.join(CSRC, source)]


def link_command(objects, out):
    return [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", out] + objects


def layers_compile_command(out):
    """The extension is host code: the host's compiler, torch's and HIP's headers."""
    from torch.utils import cpp_extension
    includes = cpp_extension.include_paths() + [os.path.join(rocm(), "include"), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", "-fvisibility=hidden",
            "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM"] + [a for i in includes for a in ("-isystem", i)] + \
           ["-o", out, os.path.join(CSRC, "layers_torch.cpp")]


def layers_link_command(obj, out):
    """Against torch's libraries (loaded before it) and the HIP library beside it."""
    from torch.utils import cpp_extension
    return [os.environ.get("CXX", "g++"), "-shared", "-o", out, obj] + \
           [f"-L{p}" for p in cpp_extension.library_paths()] + \
           ["-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_hip", f"-L{LIBDIR}", "-l:" + os.path.basename(LIB),
            "-Wl,-rpath,$ORIGIN"]


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
    """Compile the library and the extension (always recompiles, all sources side by side).  Raises on failure."""
    os.makedirs(LIBDIR, exist_ok=True)
    objects = [os.path.join(LIBDIR, s + ".o") for s in SOURCES]
    layers = os.path.join(LIBDIR, "layers_torch.cpp.o")
    commands = [compile_command(*job) for job in zip(SOURCES, objects)] + [layers_compile_command(layers)]
    with ThreadPoolExecutor(len(commands)) as ex:
        list(ex.map(lambda c: _run(c, verbose), commands))
    tmp = LIB + ".tmp"
    _run(link_command(objects, tmp), verbose)
    os.replace(tmp, LIB)
    tmp = LAYERS + ".tmp"
    _run(layers_link_command(layers, tmp), verbose)
    os.replace(tmp, LAYERS)
    for o in objects + [layers]:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
