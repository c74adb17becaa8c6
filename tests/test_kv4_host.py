"""The calls of gdn_kv4.h without a GPU: exports, documented return codes before anything is enqueued (fake,
never-dereferenced pointers), the binding's own checks, the sanitizer fuzz of the validation, and pins of the oracle."""

import ctypes
import os
import re
import shutil
import struct
import subprocess

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gated_deltanet_speculative_amd import _kv4, _lib, _round
from oracle import kv4_oracle as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_kv4.h")
HIP_INCLUDE = "/opt/rocm/include"
FAKE = 0x7F0000000000
built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")


def _p(k):
    return FAKE + k * (1 << 34)


@built
def test_exports_every_declared_function():
    names = sorted(set(re.findall(r"^(?:int|size_t)\s*(gdn_\w+)\s*\(", open(HEADER).read(), flags=re.M)))
    assert names == sorted(gdn.KV4_EXPORTED)
    lib = gdn.load_library()
    for n in names:
        assert hasattr(lib, n), n


def _shape(**kw):
    base = dict(n_seqs=2, n_nodes=4, n_slots=4, n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=20, max_pages=8,
                dtype=1)
    base.update(kw)
    return _round._CAttnShape(**base)


def _cache(first=40, **kw):
    c = dict(k=_p(first), ks=_p(first + 1), v=_p(first + 2), vs=_p(first + 3))
    c.update(kw)
    return struct.pack("4P", *[x or 0 for x in c.values()])


def _rope(sh=None, cache=None, rope=None, out=_p(9), null_shape=False):
    r = dict(inv_freq=_p(3), positions=None, pair_axis=None, n_axes=1, rot_dim=64, interleaved=0, q_norm=None, k_norm=None, eps=1e-6)
    r.update(rope or {})
    views = [struct.pack("Pqq", _p(k), 512, 64) for k in range(3)]
    return _kv4._library().gdn_rope_kv4_write(None if null_shape else ctypes.byref(sh or _shape()), 1, *views,
                                              ctypes.byref(_round._CRope(**r)), cache or _cache(), _p(6), _p(7), _p(8), None, None,
                                              out, _p(10), None)


def _attn(sh=None, cache=None, scale=0.125, mode=0, ws=_p(12), ws_bytes=1 << 30, out=_p(9), q=_p(0)):
    return _kv4._library().gdn_paged_attention_kv4(ctypes.byref(sh or _shape()), q, cache or _cache(), _p(3), _p(4), _p(5), None, None,
                                                   scale, None, mode, out, ws, ws_bytes, _p(10), None)


def _commit(sh=None, layers=2, caches=None, new_len=_p(5), status=_p(6)):
    arr = caches if caches is not None else b"".join(_cache(40 + 4 * l) for l in range(max(layers, 1)))
    return _kv4._library().gdn_kv4_commit_layers(ctypes.byref(sh or _shape()), layers, arr, _p(0), _p(1), _p(2), _p(3), None, _p(4),
                                                 new_len, status, None)


def _read(sh=None, layers=2, caches=None, k=_p(5), v=_p(6), first=_p(2)):
    arr = caches if caches is not None else b"".join(_cache(40 + 4 * l) for l in range(max(layers, 1)))
    return _kv4._library().gdn_kv4_read_layers(ctypes.byref(sh or _shape()), layers, arr, _p(0), _p(1), first, None, k, v, _p(7), None)


@built
@pytest.mark.parametrize("call", [_rope, _attn, _commit, _read])
@pytest.mark.parametrize("kw,code", [(dict(n_seqs=0), _lib.GDN_ERR_SHAPE), (dict(n_q_heads=3), _lib.GDN_ERR_SHAPE),
                                     (dict(dtype=3), _lib.GDN_ERR_SHAPE), (dict(head_dim=96), _lib.GDN_ERR_UNSUPPORTED),
                                     (dict(n_seqs=1025), _lib.GDN_ERR_UNSUPPORTED), (dict(n_pages=1 << 26), _lib.GDN_ERR_UNSUPPORTED)])
def test_shape_rejections(call, kw, code):
    assert call(_shape(**kw)) == code


@built
@pytest.mark.parametrize("call", [lambda c: _rope(cache=c), lambda c: _attn(cache=c), lambda c: _commit(layers=1, caches=c),
                                  lambda c: _read(layers=1, caches=c)])
def test_cache_rejections(call):
    for name in ("k", "ks", "v", "vs"):
        assert call(_cache(**{name: None})) == _lib.GDN_ERR_NULL
        assert call(_cache(**{name: _p(44) + 1})) == _lib.GDN_ERR_ALIGN
    assert call(_cache(k=_p(44) + 8)) == _lib.GDN_ERR_ALIGN


@built
def test_call_rejections():
    null, shape, alias, align, small, un = (_lib.GDN_ERR_NULL, _lib.GDN_ERR_SHAPE, _lib.GDN_ERR_ALIAS, _lib.GDN_ERR_ALIGN,
                                            _lib.GDN_ERR_WORKSPACE, _lib.GDN_ERR_UNSUPPORTED)
    assert _rope(null_shape=True) == null and _rope(out=None) == null and _rope(out=_p(9) + 8) == align
    assert _rope(rope=dict(rot_dim=24)) == shape and _rope(rope=dict(inv_freq=None)) == null
    for at in range(40, 44):  # the outputs among each other and against the inputs
        assert _rope(out=_p(at)) == alias
    assert _rope(cache=_cache(vs=_p(40) + 64)) == alias and _rope(cache=_cache(k=_p(0))) == alias
    assert _attn(scale=0.0) == shape and _attn(scale=3e38) == shape and _attn(mode=2) == shape and _attn(q=None) == null
    split = _shape(max_pages=100, n_pages=200)  # (1600 rows: the cache is split, and the workspace is used)
    assert _attn(split, ws_bytes=0) == small and _attn(split, ws=None) == null
    for at in range(40, 44):
        assert _attn(out=_p(at)) == alias and _attn(split, ws=_p(at)) == alias
    assert _commit(layers=0) == un and _commit(layers=65) == un and _commit(new_len=None) == null and _commit(status=None) == null
    assert _commit(caches=_cache(40) + _cache(44, v=_p(41))) == alias and _commit(new_len=_p(42)) == alias
    assert _read(layers=0) == un and _read(k=None, v=None) == null and _read(first=None) == null
    assert _read(k=_p(43)) == alias and _read(v=_p(5)) == alias and _read(k=_p(5) + 4) == align


@built
def test_workspace_size():
    sh = gdn.AttnShape(1, 1, 1, 8, 2, 128, 64, 100, 100, torch.bfloat16)
    n = gdn.paged_attention_kv4_workspace_size(sh)
    assert n > 0 and n % (4 * (128 + 2) * 8) == 0  # parts of every query row: D values, a maximum and a sum
    assert gdn.paged_attention_kv4_workspace_size(sh._replace(n_seqs=0)) == 0


@built
def test_binding_checks():
    sh = gdn.AttnShape(1, 1, 1, 2, 1, 64, 4, 2, 2, torch.float32)
    host = gdn.kv4_cache(sh, "cpu")
    assert [tuple(t.shape) for t in host] == [(2, 1, 4, 32), (2, 1, 4, 2)] * 2 and host.k.dtype == torch.uint8
    assert tuple(gdn.kv4_cache(sh, "cpu", layers=3).v_scale.shape) == (3, 2, 1, 4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.paged_attention_kv4(sh, torch.zeros(1, 1, 2, 64), host, None, None, None)
    with pytest.raises(TypeError, match="torch.Tensor"):
        gdn.rope_kv4_write(sh, None, None, None, None, host, None, None, None)
    with pytest.raises(ValueError, match="status"):
        gdn.kv4_commit_layers(sh, [host], None, None, None, None, None)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.kv4_read_layers(sh, [host], torch.zeros(1, dtype=torch.int32), None, None)


# ---------------------------------------------------------------- the oracle's pins
def test_oracle_grid_and_layout():
    """Codes by the format's words: sign, two exponent bits with bias 1, one fraction bit; the lower nibble first."""
    for code in range(16):
        e, f = (code >> 1) & 3, code & 1
        want = (1 + f / 2) * 2.0 ** (e - 1) if e else f / 2
        want = -want if code & 8 else want
        row = K.values(np.array([code | 1 << 4] + [0] * 15, np.uint8), np.array([127 + 3], np.uint8))
        assert row[0] == 8 * want and row[1] == 4.0
    assert np.isnan(K.values(np.zeros(16, np.uint8), np.array([255], np.uint8))).all()


def test_oracle_quantises_to_the_nearest_value():
    """Against a search over every value of the chosen power of two, and the choice against its words."""
    rng = np.random.default_rng(1)
    for k in range(200):
        x = rng.standard_normal(32) * 2.0 ** rng.integers(-20, 20)
        codes, scales = K.quantise(x)
        a, e = np.abs(x).max(), int(scales[0]) - 127
        assert 3.5 * 2.0 ** e <= a < 7 * 2.0 ** e  # the largest lies between 3.5 and 7 grid units
        grid = 2.0 ** e * np.array(sorted({s * m for m in K.MAGNITUDES for s in (1, -1)}))
        assert np.array_equal(np.abs(K.values(codes, scales) - x), np.abs(x[:, None] - grid).min(-1))
    assert K.nearest(2.5) == 4 and K.nearest(0.75) == 2 and K.nearest(0.25) == 0 and K.nearest(5) == 6 and K.nearest(3.5) == 6
    assert K.nearest(6.99) == K.nearest(1e30) == 7
    assert K.exponent(7.0, 125) == 1 and K.exponent(np.nextafter(7.0, 0), 125) == 0 and K.exponent(0.0, 125) == -125
    assert K.exponent(65504.0, 13) == 13 and K.exponent(3.4e38, 125) == 125 and K.exponent(1e-40, 125) == -125
    assert K.quantise(np.array([np.inf] + [1.0] * 31))[1][0] == K.quantise(np.array([np.nan] + [1.0] * 31))[1][0] == 255


# ---------------------------------------------------------------- the validation under the sanitizers
@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(HIP_INCLUDE, "hip")),
                    reason="needs g++ and the HIP headers")
def test_validation_fuzz_under_sanitizers(tmp_path):
    flags = ["-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
             "-D__HIP_PLATFORM_AMD__", "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"),
             "-I", os.path.join(ROOT, "gated_deltanet_speculative_amd", "csrc")]
    srcs = [os.path.join(ROOT, "gated_deltanet_speculative_amd", "csrc", "kv4_api.cpp"),
            os.path.join(ROOT, "tests", "host_fuzz", "kv4_harness.cpp")]
    exe = str(tmp_path / "harness")
    r = subprocess.run(["g++", *flags, *srcs, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    m = re.search(r"launches (\d+); codes:", r.stdout)
    assert m and int(m.group(1)) > 1000, r.stdout
