"""What the built kernels that several calls share hold in memory for want of registers, from the code objects in the library:
a form of a kernel for another kind of cache costs the one that was there nothing."""

import os
import re
import struct
import subprocess

import pytest

from gated_deltanet_speculative_amd import _lib

READELF = "/opt/rocm/llvm/bin/llvm-readelf"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"

# Kernel (a part of its mangled name): the most bytes of a thread's private memory and registers of the scalar file kept
# elsewhere, as these kernels had them over caches of values alone.
MOST = {"attn_pair_kernelIDF16bLb0E": (148, 2), "attn_pair_kernelIDF16_Lb0E": (156, 1), "attn_rows_kernelIDF16bLi128ELi256ELb0E": (20, 244),
        "attn_rows_kernelIDF16_Li128ELi256ELb0E": (20, 242), "attn_rows_kernelIDF16bLi128ELi64ELb0E": (0, 241),
        "attn_few_kernelIDF16bLi128ELb0E": (0, 107), "attn_few_kernelIfLi128ELb0E": (40, 22), "kv_commit_kernelILi0E": (0, 0),
        # and two forms of one kernel, neither of which costs the other anything
        "attn_pair_kernelIDF16bLb1E": (68, 1), "attn_pair_kernelIDF16_Lb1E": (76, 2)}

pytestmark = pytest.mark.skipif(not (os.path.exists(_lib.LIB_PATH) and os.path.exists(READELF)), reason="needs the library and llvm-readelf")


def _code_objects():
    """The device code objects of the library: the entries of its offload bundles."""
    data = open(_lib.LIB_PATH, "rb").read()
    at = data.find(MAGIC)
    while at >= 0:
        n, p = struct.unpack_from("<Q", data, at + len(MAGIC))[0], at + len(MAGIC) + 8
        for _ in range(n):
            offset, size, length = struct.unpack_from("<3Q", data, p)
            name = data[p + 24:p + 24 + length].decode()
            p += 24 + length
            if name.startswith("hip") and size:
                yield data[at + offset:at + offset + size]
        at = data.find(MAGIC, at + 1)


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """Mangled name: (private bytes, scalar registers elsewhere) of every kernel."""
    out, path = {}, str(tmp_path_factory.mktemp("code") / "object")
    for code in _code_objects():
        with open(path, "wb") as f:
            f.write(code)
        text = subprocess.run([READELF, "--notes", path], capture_output=True, text=True, check=True).stdout
        for part in text.split("- .agpr_count:")[1:]:
            field = lambda k: re.search(rf"\.{k}:\s+(\S+)", part)[1]  # noqa: E731
            out[field("symbol")] = int(field("private_segment_fixed_size")), int(field("sgpr_spill_count"))
    return out


@pytest.mark.parametrize("name", MOST)
def test_shared_kernels_keep_their_registers(kernels, name):
    found = [v for k, v in kernels.items() if name in k]
    assert len(found) == 1, f"{len(found)} kernels {name}"
    assert found[0][0] <= MOST[name][0] and found[0][1] <= MOST[name][1], found[0]
