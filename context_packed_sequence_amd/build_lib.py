"""Build libthdcp.so in-tree with hipcc for gfx950.

    python context_packed_sequence_amd/build_lib.py          # build
    python context_packed_sequence_amd/build_lib.py --asm    # also keep gfx950 assembly under _build/

Run it as a file (or through __graft_entry__.build()), not as a module of the
package: importing the package loads the library, which may not exist yet.

Every source is compiled on each call (the build check compiles even when a
library is already present).  Objects go to ``_build/`` beside the package; the
shared library is written next to this file and replaced atomically.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "libthdcp.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
ARCH = "gfx950"

SOURCES = ["thd_route.hip", "thd_swap.hip", "thd_roll.hip", "thd_pack.hip", "thd_stream.hip", "thd_api.hip",
           "thd_loss.hip", "thd_loss_policy.hip", "thd_loss_distill.hip", "thd_preference.hip", "thd_loss_api.hip",
           "thd_attn_plan.hip", "thd_attn_fwd.hip", "thd_attn_bwd.hip", "thd_attn_api.hip",
           "thd_embed.hip", "thd_clip.hip", "thd_params_api.hip"]

COMMON_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # no packed-FP32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE,
    "-I", CSRC,
]


def _hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the ROCm toolchain is required to build libthdcp")


def _compile(src: str, asm: bool) -> str:
    obj = os.path.join(BUILD_DIR, src + ".o")
    cmd = [_hipcc(), *COMMON_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if asm:
        cmd += ["-save-temps=obj"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    return obj


def build(verbose: bool = False, asm: bool = False) -> str:
    """Compile every source and link libthdcp.so; return its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(6, len(SOURCES))) as ex:
        objs = list(ex.map(lambda s: _compile(s, asm), SOURCES))
    tmp = LIB_PATH + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        print(f"built {LIB_PATH}")
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True, asm="--asm" in sys.argv)
