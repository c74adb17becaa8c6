"""The call of gdn_logits.h without a GPU: exports, documented return codes before anything is enqueued (fake,
never-dereferenced pointers), the binding's own checks, the sanitizer fuzz of the validation, and pins of the oracle."""

import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gated_deltanet_speculative_amd import _lib, _logits
from oracle import logits_oracle as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_logits.h")
HIP_INCLUDE = "/opt/rocm/include"
FAKE = 0x7F0000000000
built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")


def _p(k):
    return FAKE + k * (1 << 34)


@built
def test_exports_every_declared_function():
    text = open(HEADER).read()
    names = sorted(set(re.findall(r"^(?:int|size_t)\s*(gdn_\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(gdn.LOGITS_EXPORTED)
    lib = gdn.load_library()
    for n in names:
        assert hasattr(lib, n), n
    assert int(re.search(r"#define GDN_STATUS_RULE (\d+)", text).group(1)) == gdn.STATUS_RULE == L.RULE


def _call(sh=(2, 4, 4, 100, 50, 8, 1, 0), stride=100, rules=None, ptrs=None, ws_bytes=1 << 20, null_rules=False):
    u = {n: _p(20 + k) for k, (n, _) in enumerate(_logits._CLogitRules._fields_)}
    u.update(rules or {})
    a = dict(mask=_p(1), tokens=_p(2), parents=_p(3), nodes=None, slots=_p(4), out=_p(5), ws=_p(6))
    p = dict(ptrs or {})
    logits, status = p.pop("logits", _p(0)), p.pop("status", _p(7))
    a.update(p)
    shape = _logits._CLogitsShape(*sh) if sh else None
    return _logits._library().gdn_adjust_logits(ctypes.byref(shape) if sh else None, logits, stride,
                                                None if null_rules else ctypes.byref(_logits._CLogitRules(**u)), *a.values(), ws_bytes,
                                                status, None)


BASE = dict(n_seqs=2, n_nodes=4, n_slots=4, vocab=100, max_history=50, max_bias=8, dtype=1, out_dtype=0)


@built
@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), _lib.GDN_ERR_SHAPE), (dict(n_nodes=-1), _lib.GDN_ERR_SHAPE), (dict(vocab=0), _lib.GDN_ERR_SHAPE),
    (dict(max_history=-1), _lib.GDN_ERR_SHAPE), (dict(max_bias=-1), _lib.GDN_ERR_SHAPE), (dict(dtype=3), _lib.GDN_ERR_SHAPE),
    (dict(n_nodes=33), _lib.GDN_ERR_UNSUPPORTED), (dict(n_seqs=1025), _lib.GDN_ERR_UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1), _lib.GDN_ERR_UNSUPPORTED), (dict(max_history=(1 << 20) + 1), _lib.GDN_ERR_UNSUPPORTED),
    (dict(max_bias=1025), _lib.GDN_ERR_UNSUPPORTED), (dict(out_dtype=2), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_slots=1 << 28, max_history=8), _lib.GDN_ERR_UNSUPPORTED)])
def test_shape_rejections(kw, code):
    assert _call(tuple({**BASE, **kw}.values()), stride=1 << 25) == code


@built
def test_call_rejections():
    null, shape, alias, align, small = (_lib.GDN_ERR_NULL, _lib.GDN_ERR_SHAPE, _lib.GDN_ERR_ALIAS, _lib.GDN_ERR_ALIGN,
                                        _lib.GDN_ERR_WORKSPACE)
    assert _call(None) == null and _call(null_rules=True) == null
    for name in ("logits", "slots", "out", "ws"):
        assert _call(ptrs={name: None}) == null, name
    assert _call(rules=dict(history_len=None)) == null and _call(rules=dict(bias=None)) == null and _call(rules=dict(bias_tokens=None)) == null
    assert _call(stride=99) == shape and _call(stride=-100) == shape and _call(stride=1 << 41) == shape
    assert _call(ws_bytes=0) == small
    for ptr in ("logits", "mask", "tokens", "parents", "nodes", "slots", "out", "ws", "status"):
        assert _call(ptrs={ptr: _p(9) + 1}) == align, ptr
    for n, _ in _logits._CLogitRules._fields_:
        assert _call(rules={n: _p(9) + 2}) == align, n
        assert _call(rules={n: _p(5)}) == alias, n
    for ptr in ("logits", "mask", "tokens", "parents", "nodes", "slots", "status", "ws"):
        assert _call(ptrs={ptr: _p(5)}) == alias, ptr


@built
def test_workspace_size_and_binding_checks():
    sh = gdn.LogitsShape(4, 16, 4, 130001)
    n = gdn.adjust_logits_workspace_size(sh)
    assert 0 < n < 1 << 20 and n % (4 * 16 * 16) == 0
    assert gdn.adjust_logits_workspace_size(sh._replace(vocab=0)) == 0
    with pytest.raises(ValueError, match="device tensor"):
        gdn.adjust_logits(sh, torch.zeros(4, 16, 130001, dtype=torch.bfloat16), None)
    with pytest.raises(TypeError, match="dtype"):
        gdn.adjust_logits_workspace_size(sh._replace(dtype=torch.int32))


# ---------------------------------------------------------------- the oracle's pins
def test_oracle_by_hand():
    """Token 1: in the prompt; 2: three times behind it; 3: on the path; 4: biased twice; 5: not allowed."""
    rules = dict(P=1, history=np.array([[1, 2, 2, 2, 9]]), history_len=np.array([4]), prompt_len=np.array([1]), repetition=np.array([2.0]),
                 presence=np.array([0.5]), frequency=np.array([0.25]), bias_tokens=np.array([[4, 4, -1]]), bias=np.array([[1.0, 2.0, 9.0]]))
    mask = np.array([[[~(1 << 5)]] * 2], np.int32)
    res, bits = L.adjust_logits(np.full((1, 2, 8), -3.0), [0], rules, 5, mask, np.array([[3, 6]]))
    assert bits == 0
    z = res[0, 0][0]
    assert list(z) == [-3, -6, -6 - 0.75 - 0.5, -6 - 0.25 - 0.5, 0, -np.inf, -3, -3]
    assert list(res[0, 1][0][[3, 6]]) == [-6.75, -6.75]
    res, _ = L.adjust_logits(np.full((1, 2, 8), 3.0), [0], rules, 5, mask, np.array([[3, 6]]), parents=np.array([[-1, -1]]))
    assert list(res[0, 1][0]) == [3, 1.5, 1.5 - 1.25, 3, 6, -np.inf, 1.5 - 0.75, 3]  # node 1 is no child of node 0


def test_oracle_probabilities():
    z = np.array([0.0, 1.0, -np.inf, 1.0])
    e = np.exp(-1 / 0.5)
    assert np.allclose(L.probabilities(z, 0.5), np.array([e, 1, 0, 1]) / (2 + e))
    assert list(L.probabilities(z, 0.0)) == [0, 1, 0, 0] and list(L.probabilities(np.array([np.nan, 3.0]), 0.0)) == [0, 1]
    assert np.isnan(L.probabilities(np.array([np.nan, 3.0]), 1.0)).all() and not L.probabilities(np.full(3, -np.inf), 1.0).any()
    assert list(L.probabilities(np.array([np.inf, 3.0, np.inf]), 1.0)) == [0.5, 0, 0.5]


# ---------------------------------------------------------------- the validation under the sanitizers
@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(HIP_INCLUDE, "hip")),
                    reason="needs g++ and the HIP headers")
def test_validation_fuzz_under_sanitizers(tmp_path):
    flags = ["-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"),
             "-I", os.path.join(ROOT, "gated_deltanet_speculative_amd", "csrc")]
    srcs = [os.path.join(ROOT, "gated_deltanet_speculative_amd", "csrc", "logits_api.cpp"),
            os.path.join(ROOT, "tests", "host_fuzz", "logits_harness.cpp")]
    exe = str(tmp_path / "harness")
    r = subprocess.run(["g++", *flags, *srcs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    m = re.search(r"launches (\d+); codes:", r.stdout)
    assert m and int(m.group(1)) > 1000, r.stdout
