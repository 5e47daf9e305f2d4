"""Compile the HIP library for gfx950 (in-tree, no JIT cache)."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SOURCES = [os.path.join(CSRC, f) for f in ("spec_verify.hip", "sv_rules.hip", "sv_head.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libspec_verify.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed-fp32 instructions stay off: plain fp32 arithmetic only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def _run(cmd) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def build(verbose: bool = False) -> str:
    """Compile every source (side by side) and link them into one library."""
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SOURCES]
        said = list(pool.map(lambda so: _run([HIPCC, *FLAGS, "-I", INCLUDE, "-c", so[0], "-o", so[1]]),
                             zip(SOURCES, objects)))
        out = LIB + ".tmp"
        said.append(_run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objects, "-o", out]))
    if verbose and any(said):
        print("".join(said))
    os.replace(out, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
