"""Build libgdnverify.so (the C-ABI library) for gfx950 with hipcc, in-tree.

    python -m gated_deltanet_speculative_amd.build [--library]

Compiles every source under csrc/ to an object in _build/ and links the shared
library next to this file, and beside it the Python binding's tensor checks (_marshal.so),
unless --library is given.  Always recompiles (cheap: a few seconds per file).  The library
needs hipcc alone; the tensor checks need g++ and the headers of Python and torch.
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
MARSHAL = os.path.join(PKG, "_marshal.so")
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


def _build_marshal() -> str:
    """The binding's tensor checks as a Python extension (host code only, against torch's headers)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    includes = [a for d in (*ext.include_paths(), sysconfig.get_paths()["include"]) for a in ("-isystem", d)]
    libs = [a for d in ext.library_paths() for a in (f"-L{d}", f"-Wl,-rpath,{d}")]
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *includes, os.path.join(CSRC, "marshal.cpp"), "-o", tmp, *libs, "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    return MARSHAL


def _link(objs: list) -> None:
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(verbose: bool = True, binding: bool = True) -> str:
    """Builds the library and, with `binding`, the tensor checks; the library is there before a failure of the
    latter is raised."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(4, len(SOURCES))) as ex:
        marshal = ex.submit(_build_marshal) if binding else None
        _link(list(ex.map(_compile, SOURCES)))
    if verbose:
        print(f"built {LIB}")
    if marshal:
        try:
            marshal.result()
        except Exception as e:
            raise RuntimeError(f"{LIB} is built, the Python binding's {os.path.basename(MARSHAL)} is not: {e}") from e
    return LIB


if __name__ == "__main__":
    build(binding="--library" not in sys.argv[1:])
    sys.exit(0)
