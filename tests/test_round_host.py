"""The calls of gdn_round.h without a GPU: exports, documented return codes before anything is
enqueued (fake, never-dereferenced pointers), the sanitizer fuzz of the validation, the binding's own
checks, and pins of the fp64 oracle."""

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
from gated_deltanet_speculative_amd import _lib, _round
from oracle import round_oracle as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gdn_round.h")
HIP_INCLUDE = "/opt/rocm/include"
FAKE = 0x7F0000000000
built = pytest.mark.skipif(not os.path.exists(_lib.LIB_PATH), reason="library not built")


def _p(k):
    return FAKE + k * (1 << 34)


@built
def test_exports_every_declared_function():
    names = sorted(set(re.findall(r"^(?:int|size_t)\s*(gdn_\w+)\s*\(", open(HEADER).read(), flags=re.M)))
    assert names == sorted(gdn.ROUND_EXPORTED)
    lib = gdn.load_library()
    for n in names:
        assert hasattr(lib, n), n


def test_constants_match_the_header():
    text = open(HEADER).read()
    value = lambda n: int(re.search(rf"#define {n} (\d+)", text).group(1))  # noqa: E731
    assert value("GDN_STATUS_LENGTH") == gdn.STATUS_LENGTH == R.LENGTH
    assert value("GDN_STATUS_PAGE") == gdn.STATUS_PAGE == R.PAGE
    assert value("GDN_STATUS_TOKEN") == gdn.STATUS_TOKEN == R.TOKEN
    assert value("GDN_STATUS_AXIS") == gdn.STATUS_AXIS == R.AXIS
    assert [value(f"GDN_DTYPE_{n}") for n in ("F32", "BF16", "F16")] == [
        _round.DTYPES[d] for d in (torch.float32, torch.bfloat16, torch.float16)]


def _shape(**kw):
    base = dict(n_seqs=2, n_nodes=4, n_slots=4, n_q_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=20, max_pages=8,
                dtype=1)
    base.update(kw)
    return _round._CAttnShape(**base)


def _rope(sh=None, x_dtype=1, views=None, rope=None, ptrs=None):
    v = views or [(_p(0), 512, 64), (_p(1), 512, 64), (_p(2), 512, 64)]
    r = dict(inv_freq=_p(3), positions=None, pair_axis=None, n_axes=1, rot_dim=64, interleaved=0, q_norm=None, k_norm=None, eps=1e-6)
    r.update(rope or {})
    a = dict(k=_p(4), v=_p(5), slot=_p(6), table=_p(7), len=_p(8), parents=None, nodes=None, out=_p(9), status=_p(10))
    a.update(ptrs or {})
    return _round._library().gdn_rope_kv_write(ctypes.byref(sh or _shape()), x_dtype, *[struct.pack("Pqq", x[0] or 0, *x[1:]) for x in v],
                                               ctypes.byref(_round._CRope(**r)), *a.values(), None)


def _attn(sh=None, scale=0.125, gate=None, mode=0, ws=_p(12), ws_bytes=1 << 30, ptrs=None):
    a = dict(q=_p(0), k=_p(1), v=_p(2), slot=_p(3), table=_p(4), len=_p(5), parents=None, nodes=None)
    out, status = _p(9), _p(10)
    p = dict(ptrs or {})
    out, status = p.pop("out", out), p.pop("status", status)
    a.update(p)
    g = None if gate is None else struct.pack("Pqq", gate[0] or 0, *gate[1:])
    return _round._library().gdn_paged_attention(ctypes.byref(sh or _shape()), *a.values(), scale, g, mode, out, ws, ws_bytes, status, None)


def _commit(sh=None, layers=2, k=None, v=None, ptrs=None):
    k, v = k or [_p(20 + 2 * i) for i in range(layers)], v or [_p(21 + 2 * i) for i in range(layers)]
    a = dict(slot=_p(0), table=_p(1), len=_p(2), parents=_p(3), nodes=None, accept=_p(4), new_len=_p(5), status=_p(6))
    a.update(ptrs or {})
    arr = ctypes.c_void_p * max(len(k), 1)
    return _round._library().gdn_kv_commit_layers(ctypes.byref(sh or _shape()), layers, arr(*k), arr(*v), *a.values(), None)


def _accept(sh=(2, 4, 100, 0), ptrs=None, ws_bytes=1 << 20):
    a = dict(target=_p(0), root=None, draft=None, tokens=_p(1), parents=None, nodes=None, slots=None, u=_p(2), un=_p(3), node=_p(4),
             count=_p(5), next=_p(6), ws=_p(7))
    a.update(ptrs or {})
    return _round._library().gdn_draft_accept(ctypes.byref(_round._CAcceptShape(*sh)), *a.values(), ws_bytes, None, None)


@built
@pytest.mark.parametrize("kw,code", [
    (dict(n_seqs=0), _lib.GDN_ERR_SHAPE),
    (dict(n_nodes=-1), _lib.GDN_ERR_SHAPE),
    (dict(n_q_heads=3), _lib.GDN_ERR_SHAPE),
    (dict(page_size=0), _lib.GDN_ERR_SHAPE),
    (dict(dtype=3), _lib.GDN_ERR_SHAPE),
    (dict(head_dim=96), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_seqs=1025), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_nodes=65537), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_q_heads=1026), _lib.GDN_ERR_UNSUPPORTED),
    (dict(page_size=65537), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_pages=1 << 26), _lib.GDN_ERR_UNSUPPORTED),
    (dict(max_pages=(1 << 26) + 1), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_slots=1 << 28), _lib.GDN_ERR_UNSUPPORTED),
    (dict(n_seqs=1024, n_nodes=65536, n_q_heads=6), _lib.GDN_ERR_UNSUPPORTED),  # C N H_q = 1.5 * 2^28
])
def test_shape_rejections(kw, code):
    assert _rope(_shape(**kw)) == code
    assert _attn(_shape(**kw)) == code
    assert _commit(_shape(**kw), ptrs=dict(parents=None)) == code
    assert _round._library().gdn_paged_attention_workspace_size(ctypes.byref(_shape(**kw))) == 0


@built
def test_trees_are_bounded():
    sh = _shape(n_nodes=33)
    assert _rope(sh, ptrs=dict(parents=_p(15))) == _attn(sh, ptrs=dict(parents=_p(15))) == _commit(sh) == _lib.GDN_ERR_UNSUPPORTED


@built
def test_rope_rejections():
    for ptr in ("k", "v", "slot", "table", "len", "out"):
        assert _rope(ptrs={ptr: None}) == _lib.GDN_ERR_NULL, ptr
    assert _rope(rope=dict(inv_freq=None)) == _lib.GDN_ERR_NULL
    assert _rope(views=[(None, 512, 64), (_p(1), 512, 64), (_p(2), 512, 64)]) == _lib.GDN_ERR_NULL
    for bad in (dict(rot_dim=24), dict(rot_dim=0), dict(rot_dim=80), dict(interleaved=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(n_axes=0), dict(n_axes=2)):
        assert _rope(rope=bad) == _lib.GDN_ERR_SHAPE, bad
    assert _rope(x_dtype=5) == _lib.GDN_ERR_SHAPE
    assert _rope(x_dtype=2) == _lib.GDN_ERR_UNSUPPORTED  # float16 values into a bfloat16 cache
    assert _rope(rope=dict(n_axes=17, positions=_p(11))) == _lib.GDN_ERR_UNSUPPORTED
    ok = [(_p(0), 512, 64), (_p(1), 512, 64), (_p(2), 512, 64)]
    for k, bad, code in ((0, (_p(0), 516, 64), _lib.GDN_ERR_ALIGN), (1, (_p(1), 512, 4), _lib.GDN_ERR_ALIGN),
                         (2, (_p(2) + 8, 512, 64), _lib.GDN_ERR_ALIGN), (0, (_p(0), -512, 64), _lib.GDN_ERR_SHAPE),
                         (0, (_p(9), 512, 64), _lib.GDN_ERR_ALIAS), (2, (_p(5), 512, 64), _lib.GDN_ERR_ALIAS)):
        assert _rope(views=[*ok[:k], bad, *ok[k + 1:]]) == code, bad
    assert _rope(ptrs=dict(v=_p(4))) == _lib.GDN_ERR_ALIAS  # one buffer for both caches
    assert _rope(rope=dict(inv_freq=_p(3) + 4)) == _lib.GDN_ERR_ALIGN
    assert _rope(ptrs=dict(table=_p(7) + 2)) == _lib.GDN_ERR_ALIGN


@built
def test_attention_rejections():
    for ptr in ("q", "k", "v", "slot", "table", "len", "out"):
        assert _attn(ptrs={ptr: None}) == _lib.GDN_ERR_NULL, ptr
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _attn(scale=scale) == _lib.GDN_ERR_SHAPE
    assert _attn(mode=2) == _lib.GDN_ERR_SHAPE
    assert _attn(gate=(None, 256, 64)) == _lib.GDN_ERR_NULL
    assert _attn(gate=(_p(13), 256, 60)) == _lib.GDN_ERR_ALIGN
    assert _attn(gate=(_p(9), 256, 64)) == _lib.GDN_ERR_ALIAS
    assert _attn(ptrs=dict(q=_p(0) + 8)) == _lib.GDN_ERR_ALIGN
    assert _attn(ptrs=dict(out=_p(2))) == _lib.GDN_ERR_ALIAS
    sh = _shape(max_pages=1000)
    need = _round._library().gdn_paged_attention_workspace_size(ctypes.byref(sh))
    assert need > 0
    assert _attn(sh, ws_bytes=need - 1) == _lib.GDN_ERR_WORKSPACE
    assert _attn(sh, ws=None) == _lib.GDN_ERR_NULL
    assert _attn(sh, ws=_p(12) + 4) == _lib.GDN_ERR_ALIGN
    assert _attn(sh, ws=_p(1)) == _lib.GDN_ERR_ALIAS


@built
def test_accept_rejections():
    for ptr in ("target", "tokens", "node", "count", "next", "ws", "u", "un"):
        assert _accept(ptrs={ptr: None}) == _lib.GDN_ERR_NULL, ptr
    for sh, code in (((0, 4, 100, 0), 2), ((2, 0, 100, 0), 2), ((2, 4, 0, 0), 2), ((2, 4, 100, 9), 2), ((1025, 4, 100, 0), 3),
                     ((2, 33, 100, 0), 3), ((2, 4, (1 << 24) + 1, 0), 3)):
        assert _accept(sh) == code
        assert _round._library().gdn_draft_accept_workspace_size(ctypes.byref(_round._CAcceptShape(*sh))) == 0
    assert _accept(ptrs=dict(draft=_p(8), parents=_p(9))) == _lib.GDN_ERR_UNSUPPORTED
    assert _accept(ptrs=dict(draft=_p(8), u=None, un=None)) == _lib.GDN_ERR_UNSUPPORTED
    assert _accept(ws_bytes=8) == _lib.GDN_ERR_WORKSPACE
    assert _accept(ptrs=dict(target=_p(0) + 2)) == _lib.GDN_ERR_ALIGN
    assert _accept(ptrs=dict(ws=_p(7) + 8)) == _lib.GDN_ERR_ALIGN
    assert _accept(ptrs=dict(count=_p(4))) == _lib.GDN_ERR_ALIAS
    assert _accept(ptrs=dict(next=_p(1))) == _lib.GDN_ERR_ALIAS


@built
def test_commit_rejections():
    for ptr in ("slot", "table", "len", "accept", "new_len", "status"):
        assert _commit(ptrs={ptr: None}) == _lib.GDN_ERR_NULL, ptr
    assert _commit(layers=0) == _commit(layers=65, k=[_p(20)] * 65, v=[_p(21)] * 65) == _lib.GDN_ERR_UNSUPPORTED
    assert _commit(k=[_p(20), None]) == _lib.GDN_ERR_NULL
    assert _commit(k=[_p(20), _p(20)]) == _commit(v=[_p(20), _p(23)]) == _commit(k=[_p(5), _p(22)]) == _lib.GDN_ERR_ALIAS
    assert _commit(ptrs=dict(new_len=_p(2))) == _lib.GDN_ERR_ALIAS
    assert _commit(k=[_p(20) + 8, _p(22)]) == _lib.GDN_ERR_ALIGN


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.exists(os.path.join(HIP_INCLUDE, "hip")),
                    reason="needs g++ and the HIP headers")
def test_validation_fuzz_under_sanitizers(tmp_path):
    csrc, fuzz = os.path.join(ROOT, "gated_deltanet_speculative_amd", "csrc"), os.path.join(ROOT, "tests", "host_fuzz")
    flags = ["-O1", "-g", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
             "-I", HIP_INCLUDE, "-I", os.path.join(ROOT, "include"), "-I", csrc]
    exe = str(tmp_path / "harness")
    r = subprocess.run(["g++", *flags, os.path.join(csrc, "round_api.cpp"), os.path.join(fuzz, "round_stubs.cpp"),
                        os.path.join(fuzz, "round_harness.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, (r.stdout + r.stderr)[-3000:]
    m = re.search(r"launches (\d+); codes:", r.stdout)
    assert m and int(m.group(1)) > 1000, r.stdout


def test_binding_refuses_host_tensors_and_wrong_types():
    sh = gdn.AttnShape(1, 1, 1, 2, 1, 64, 16, 2, 2, torch.float32)
    t = torch.zeros
    i = lambda *s: t(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        gdn.paged_attention(sh, t(1, 1, 2, 64), t(sh.cache_shape), t(sh.cache_shape), i(1), i(1, 2), i(1))
    with pytest.raises(TypeError):
        gdn.paged_attention(sh, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="device tensor"):
        gdn.draft_accept(gdn.AcceptShape(1, 1, 5), t(1, 1, 5), i(1, 1))
    with pytest.raises(ValueError, match="device tensor"):
        gdn.rope_kv_write(sh, t(1, 1, 2, 64), t(1, 1, 1, 64), t(1, 1, 1, 64), t(32, dtype=torch.float64), None, None, None, None, None)
    with pytest.raises(ValueError, match="status"):
        gdn.kv_commit_layers(sh, [], [], None, None, None, None, None)
    with pytest.raises(TypeError, match="dtype"):
        sh._replace(dtype=torch.int8).c_struct()


@built
def test_binding_survives_tensors_without_storage():
    """A tensor that only pretends to be on a device raises; the process goes on."""
    from torch._subclasses.fake_tensor import FakeTensorMode

    sh = gdn.AcceptShape(1, 1, 5)
    with FakeTensorMode():
        fake = torch.empty(1, 1, 5, device="meta")
    with pytest.raises((ValueError, TypeError, RuntimeError)):
        gdn.draft_accept(sh, fake, torch.zeros(1, 1, dtype=torch.int32))
    for t, shape in ((torch.empty(3, device="meta"), (3,)), (torch.zeros(3).to_sparse(), (3,)), (torch.zeros(3), (4,)), ("no", (3,))):
        with pytest.raises((ValueError, TypeError)):
            _round._ptr(t, "t", torch.float32, shape, 0)
    with pytest.raises(TypeError):
        _round._ptr(torch.zeros(3), "t", torch.float32)


# ---------------------------------------------------------------- pins of the oracle
def test_oracle_attention_closed_forms():
    """Equal keys average the attended values; one attended row is its value; a tree node is its path's chain."""
    rng = np.random.default_rng(0)
    page, Hkv, D = 4, 2, 8
    k, v = np.ones((6, Hkv, page, D)), rng.standard_normal((6, Hkv, page, D))
    table, length, slots = np.array([[5, 0, 2]], np.int32), np.array([3], np.int32), np.array([0], np.int32)
    q = rng.standard_normal((1, 4, 4, D))
    flat = v[[5, 0, 2]].transpose(0, 2, 1, 3).reshape(12, Hkv, D)  # the lane's rows in order
    res, bits = R.paged_attention(q, k, v, slots, table, length)
    assert bits == 0
    for i in range(4):
        for h in range(4):
            assert np.allclose(res[0, i][0][h], flat[:3 + i + 1, h // 2].mean(0))
    parents = np.array([[-1, 0, 0, 2]], np.int32)
    res, _ = R.paged_attention(q, k, v, slots, table, length, parents)
    assert np.allclose(res[0, 3][0][0], flat[[0, 1, 2, 3, 5, 6], 0].mean(0))
    res, _ = R.paged_attention(q, k, v, slots, table, np.array([0], np.int32))
    assert np.allclose(res[0, 0][0][1], flat[0, 0])
    k = rng.standard_normal(k.shape)
    chain, _ = R.paged_attention(q, k, v, slots, table, length)
    tree, _ = R.paged_attention(q, k, v, slots, table, length, np.array([[-1, 0, 1, 2]], np.int32))
    assert all(np.array_equal(chain[0, i][0], tree[0, i][0]) for i in range(4))


def test_oracle_rotation_keeps_relative_positions():
    """q.k after the rotation depends on the positions' difference only; norms are kept; angle zero changes nothing."""
    rng = np.random.default_rng(1)
    q, k, inv = rng.standard_normal(16), rng.standard_normal(16), 100.0 ** (-np.arange(6) / 6)
    for inter in (False, True):
        dot = lambda a, b: R.rotate(q, a * inv, inter) @ R.rotate(k, b * inv, inter)  # noqa: E731
        assert abs(dot(7, 3) - dot(104, 100)) < 1e-10
        assert abs(np.linalg.norm(R.rotate(q, 9 * inv, inter)) - np.linalg.norm(q)) < 1e-12
        assert np.array_equal(R.rotate(q, 0 * inv, inter), q)
    quarter = R.rotate(np.array([1.0, 0.0, 5.0]), np.array([np.pi / 2]), False)
    assert np.allclose(quarter, [0, 1, 5])


def test_oracle_acceptance_leaves_the_targets_distribution():
    """Exact integration over the random numbers: the first token's distribution is the target's, for a drawn draft
    and for candidates (whichever they are)."""
    p, q = np.array([0.5, 0.2, 0.2, 0.1]), np.array([0.1, 0.6, 0.1, 0.2])
    n = 400
    grid = (np.arange(n) + 0.5) / n
    share = np.zeros(4)
    for t in range(4):
        for u in grid:
            if u * q[t] < p[t]:
                share[t] += q[t] / n
            else:
                w = np.maximum(p - q, 0)
                share += q[t] / n * w / w.sum()
    assert np.abs(share - p).max() <= 1 / n
    for cand in ([2, 0], [3, 1], [1, 1]):
        share = np.zeros(4)
        for u0 in grid[::8]:
            for u1 in grid[::8]:
                for w in grid[::40]:
                    res, _ = R.draft_accept(np.tile(p, (1, 2, 1)), [cand], root=p[None], parents=np.array([[-1, -1]]),
                                            u_accept=np.array([[u0, u1]]), u_next=np.array([w]))
                    node, _, token = res[0]
                    share[cand[node] if node >= 0 else token] += 1
        assert np.abs(share / share.sum() - p).max() <= 0.11  # (ten values of u_next: a step of 0.1)


def test_oracle_commit_equals_sequential_moves():
    rng = np.random.default_rng(2)
    parents = np.array([[-1, 0, 0, 1, 3]], np.int32)
    table, length, slots = np.array([[2, 0, 1]], np.int32), np.array([3], np.int32), np.array([0], np.int32)
    for e in range(-1, 5):
        k, v = rng.standard_normal((3, 1, 4, 2)), rng.standard_normal((3, 1, 4, 2))
        flat = k[[2, 0, 1]].reshape(12, 2).copy()
        new_len, bits = R.kv_commit([k], [v], slots, table, length, np.array([e]), parents)
        path = R.path_of(parents[0], e) if e >= 0 else []
        assert bits == 0 and new_len[0] == 3 + len(path)
        assert np.array_equal(k[[2, 0, 1]].reshape(12, 2)[3:3 + len(path)], flat[[3 + a for a in path]])
