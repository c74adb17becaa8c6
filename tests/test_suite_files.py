"""Every GPU test file is collected with the tests it has (a renamed or unregistered file must not drop out of the run
unnoticed because the others are many)."""

import collections
import os
import subprocess
import sys

from conftest import ROOT

GPU_TESTS = {"test_gpu_acceptance.py": 15, "test_gpu_attention_numerics.py": 231, "test_gpu_bench.py": 4, "test_gpu_decode.py": 29,
             "test_gpu_edges.py": 100, "test_gpu_paged_attention.py": 221, "test_gpu_parity.py": 71, "test_gpu_prefill.py": 14,
             "test_gpu_ragged.py": 17, "test_gpu_round.py": 183, "test_zz_no_alloc.py": 2}


def test_every_gpu_file_is_collected():
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(ROOT, "tests"), "--collect-only", "-q", "-m", "gpu", "-p",
                        "no:cacheprovider"], capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    n = collections.Counter(os.path.basename(line.split("::")[0]) for line in r.stdout.splitlines() if "::" in line)
    short = {f: (n[f], least) for f, least in GPU_TESTS.items() if n[f] < least}
    assert not short, f"GPU tests collected, expected: {short}"
