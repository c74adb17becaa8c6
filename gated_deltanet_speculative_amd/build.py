"""Build libgdnverify.so (the C-ABI library) for gfx950 with hipcc, in-tree.

    python -m gated_deltanet_speculative_amd.build

Compiles every source under csrc/ to an object in _build/ and links the shared
library next to this file.  Always recompiles (cheap: a few seconds per file).
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdnverify.so")
ARCH = "gfx950"

SOURCES = ["gdn_api.cpp", "conv_tree_step.hip", "tree_verify.hip", "replay_commit.hip", "decode_step.hip",
           "prefill.hip", "round_api.cpp", "rope_kv_write.hip", "paged_attention.hip", "draft_accept.hip",
           "kv_commit.hip"]

# Packed-FP32 instructions are disabled: the compiler may otherwise fuse ordinary
# float code into them.
HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    return "hipcc"


# Per-source additions.  The prefill's state kernel keeps its state tile as MFMA
# accumulators across a loop that also scales it on the VALU; in the accumulator-register
# form every chunk moves the tile between register files (about 140 moves per chunk),
# which the VGPR form of the MFMA instructions avoids (6% faster prefill, bit-identical).
SOURCE_FLAGS = {"prefill.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *HIPCC_FLAGS, *SOURCE_FLAGS.get(src, []), "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(4, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
