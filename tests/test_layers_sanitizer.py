"""Host code of the MX8, activation, norm and join entry points under
AddressSanitizer and UndefinedBehaviorSanitizer (tests/sanitize/layers_checks.cpp).
Device code is compiled as usual and never runs.  The executable is kept under
tests/sanitize/layers/_build by the sources' digest."""
import hashlib
import os
import shutil
import subprocess

import pytest

from inverse_root_preconditioning_amd import build as B

HERE = os.path.dirname(os.path.abspath(__file__))
DRIVER = os.path.join(HERE, "sanitize", "layers_checks.cpp")
OUTDIR = os.path.join(HERE, "sanitize", "layers", "_build")
SOURCES = [os.path.join(B.CSRC, s) for s in ("layers.hip", "norm.hip")]
FLAGS = ["--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
         "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
         "-Xarch_host", "-fno-sanitize-recover=undefined",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def _digest():
    h = hashlib.sha256(" ".join(FLAGS).encode())
    paths = [DRIVER, os.path.join(B.ROOT, "include", "shampoo.h")] + SOURCES
    paths += [os.path.join(B.CSRC, x) for x in B.HEADERS]
    for p in paths:
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


@pytest.mark.skipif(not os.path.exists(B.hipcc()), reason="hipcc not available")
def test_layer_host_code_under_sanitizers():
    exe = os.path.join(OUTDIR, f"layers_{_digest()}")
    if not os.path.exists(exe):
        if os.path.isdir(OUTDIR):
            shutil.rmtree(OUTDIR)
        os.makedirs(OUTDIR)
        cmd = [B.hipcc()] + FLAGS + ["-I", os.path.join(B.ROOT, "include"), DRIVER] + SOURCES + ["-o", exe + ".tmp"]
        res = subprocess.run(cmd, capture_output=True, text=True, timeout=1200)
        assert res.returncode == 0, res.stderr[-4000:]
        os.replace(exe + ".tmp", exe)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0:exitcode=23",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert res.returncode == 0, (res.returncode, res.stdout[-2000:], res.stderr[-6000:])
    assert "layer checks passed" in res.stdout
