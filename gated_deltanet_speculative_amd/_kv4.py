"""ctypes binding of the gdn_kv4.h calls: the attention layers' part of a round over a cache held in 4 bits.

Argument marshalling only, as in the binding of the gdn_round.h calls, whose helpers and shapes it uses.  There is no
fallback.
"""

from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple

import torch

from . import _round as R
from ._lib import MAX_LAYERS, load_library

KV4_EXPORTED = ("gdn_rope_kv4_write", "gdn_paged_attention_kv4", "gdn_paged_attention_kv4_workspace_size",
                "gdn_kv4_commit_layers", "gdn_kv4_read_layers")

_i32, _vp = ctypes.c_int32, ctypes.c_void_p


class Kv4Cache(NamedTuple):
    """One layer's cache, or every layer's with a leading layer axis: uint8 tensors of codes
    [n_pages, H_kv, page_size, D / 2] and of scales [n_pages, H_kv, page_size, D / 32]."""

    k: torch.Tensor
    k_scale: torch.Tensor
    v: torch.Tensor
    v_scale: torch.Tensor


def kv4_cache(sh: R.AttnShape, device="cuda", layers=None) -> Kv4Cache:
    """A cache of zeros for this shape (with `layers`, of that many layers in one tensor each)."""
    lead = () if layers is None else (layers,)
    make = lambda fill, step: torch.full((*lead, *sh.cache_shape[:3], sh.head_dim // step), fill, dtype=torch.uint8,  # noqa: E731
                                         device=device)
    return Kv4Cache(make(0, 2), make(127, 32), make(0, 2), make(127, 32))


_calls = None


def _library():
    """The library with the prototypes of these calls (looked up once)."""
    global _calls
    if _calls is None:
        lib = load_library()
        sp = ctypes.POINTER(R._CAttnShape)
        lib.gdn_rope_kv4_write.argtypes = [sp, _i32, _vp, _vp, _vp, ctypes.POINTER(R._CRope)] + [_vp] * 9
        lib.gdn_paged_attention_kv4.argtypes = [sp] + [_vp] * 7 + [ctypes.c_float, _vp, _i32, _vp, _vp, ctypes.c_size_t, _vp, _vp]
        lib.gdn_paged_attention_kv4_workspace_size.argtypes = [sp]
        lib.gdn_kv4_commit_layers.argtypes = [sp, _i32] + [_vp] * 10
        lib.gdn_kv4_read_layers.argtypes = [sp, _i32] + [_vp] * 9
        for f in ("gdn_rope_kv4_write", "gdn_paged_attention_kv4", "gdn_kv4_commit_layers", "gdn_kv4_read_layers"):
            getattr(lib, f).restype = _i32
        lib.gdn_paged_attention_kv4_workspace_size.restype = ctypes.c_size_t
        _calls = lib
    return _calls


_four = struct.Struct("4P").pack


def _pointers(cache, sh, device, lead=()) -> list:
    """Addresses of the four tensors of a Kv4Cache, in the order of gdn_kv4_cache."""
    if not isinstance(cache, Kv4Cache):
        raise TypeError("the cache must be a Kv4Cache")
    codes = (*lead, sh.n_pages, sh.n_kv_heads, sh.page_size, sh.head_dim // 2)
    scales = (*codes[:-1], sh.head_dim // 32)
    return [R._ptr(cache.k, "cache.k", torch.uint8, codes, device), R._ptr(cache.k_scale, "cache.k_scale", torch.uint8, scales, device),
            R._ptr(cache.v, "cache.v", torch.uint8, codes, device), R._ptr(cache.v_scale, "cache.v_scale", torch.uint8, scales, device)]


def _layers(caches, sh, device, name) -> tuple:
    """(number of layers, gdn_kv4_cache array as bytes) of one Kv4Cache with a leading layer axis, or of a sequence."""
    if isinstance(caches, Kv4Cache):
        n = caches.k.shape[0] if isinstance(caches.k, torch.Tensor) and caches.k.dim() else 0
        step = sh.n_pages * sh.n_kv_heads * sh.page_size * sh.head_dim
        base = _pointers(caches, sh, device, (n,)) if n else []
        flat = [p + i * (step // (32 if j % 2 else 2)) for i in range(n) for j, p in enumerate(base)]
    else:
        flat = [p for c in caches for p in _pointers(c, sh, device)]
        n = len(flat) // 4
    if not 1 <= n <= MAX_LAYERS:
        raise ValueError(f"{name}: {n} layers, expected 1..{MAX_LAYERS}")
    return n, struct.pack(f"{4 * n}P", *flat)


def rope_kv4_write(sh: R.AttnShape, q, k, v, inv_freq, cache, slot_ids, page_table, seq_len, positions=None, pair_axis=None,
                   parents=None, lane_nodes=None, q_norm=None, k_norm=None, eps=1e-6, interleaved=False, q_out=None,
                   status=None):
    """Rotary positions of q and k and the write of k and v, quantised to 4 bits, into the slots' pages behind their
    committed rows: rope_kv_write with a Kv4Cache in the place of the two caches.  Returns (q_out, status)."""
    device = R._device(q, "q")
    q_out, status, lead, tail = R._rope_arguments(sh, q, k, v, inv_freq, slot_ids, page_table, seq_len, positions, pair_axis,
                                                  parents, lane_nodes, q_norm, k_norm, eps, interleaved, q_out, status, device)
    R._call(device, _library().gdn_rope_kv4_write, "gdn_rope_kv4_write", *lead, _four(*_pointers(cache, sh, device)), *tail)
    return q_out, status


def paged_attention_kv4_workspace_size(sh: R.AttnShape) -> int:
    """Bytes of device workspace paged_attention_kv4 needs for this shape (0 for an invalid shape)."""
    return int(_library().gdn_paged_attention_kv4_workspace_size(ctypes.byref(R._cs(sh))))


def paged_attention_kv4(sh: R.AttnShape, q, cache, slot_ids, page_table, seq_len, parents=None, lane_nodes=None, scale=None,
                        gate=None, gate_mode=1, out=None, workspace=None, status=None):
    """Attention of the round's tokens over a 4-bit cache: paged_attention with a Kv4Cache in the place of the two
    caches (`workspace` is at least paged_attention_kv4_workspace_size(sh) bytes).  Returns (out, status)."""
    device = R._device(q, "q")
    shape = (sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim)
    if out is None:
        out = torch.empty(shape, dtype=sh.dtype, device=device)
    status = R._status_word(status, device)
    lib, cs = _library(), ctypes.byref(R._cs(sh))
    if workspace is None:
        workspace = torch.empty(max(lib.gdn_paged_attention_kv4_workspace_size(cs) // 4, 1), dtype=torch.float32, device=device)
    else:
        workspace = R._scratch(workspace, device)
    R._call(device, lib.gdn_paged_attention_kv4, "gdn_paged_attention_kv4", cs, R._ptr(q, "q", sh.dtype, shape, device),
            _four(*_pointers(cache, sh, device)), *R._places(sh, slot_ids, page_table, seq_len, device),
            *R._tree(sh, parents, lane_nodes, device), 1.0 / math.sqrt(sh.head_dim) if scale is None else scale,
            None if gate is None else R._view(gate, "gate", sh.dtype, shape, device), int(gate_mode),
            R._ptr(out, "out", sh.dtype, shape, device), workspace.data_ptr(), workspace.numel() * 4, status.data_ptr())
    return out, status


def kv4_commit_layers(sh: R.AttnShape, caches, slot_ids, page_table, seq_len, accept_node, status, parents=None,
                      lane_nodes=None, new_len=None):
    """Moves the accepted paths' rows of every layer's 4-bit cache together behind the committed rows and returns the
    new lengths [P]: kv_commit_layers with a Kv4Cache of tensors with a leading layer axis, or a sequence of one
    Kv4Cache a layer.  A transaction on the status word: every lane and layer, or nothing."""
    if status is None:
        raise ValueError("kv4_commit_layers needs a status word (the round's transaction flag)")
    device = R._device(status, "status")
    if new_len is None:
        new_len = torch.empty(sh.n_slots, dtype=torch.int32, device=device)
    n, arrays = _layers(caches, sh, device, "kv4_commit_layers")
    R._call(device, _library().gdn_kv4_commit_layers, "gdn_kv4_commit_layers", ctypes.byref(R._cs(sh)), n, arrays,
            *R._places(sh, slot_ids, page_table, seq_len, device), *R._tree(sh, parents, lane_nodes, device),
            R._ptr(accept_node, "accept_node", torch.int32, (sh.n_seqs,), device),
            R._ptr(new_len, "new_len", torch.int32, (sh.n_slots,), device),
            R._ptr(status, "status", torch.int32, (1,), device))
    return new_len


def kv4_read_layers(sh: R.AttnShape, caches, slot_ids, page_table, first_row, lane_nodes=None, k_out=None, v_out=None,
                    status=None):
    """Rows first_row[c] .. first_row[c] + N - 1 of every lane's slot as values of sh.dtype, for every layer (caches as in
    kv4_commit_layers).  Returns (k_out, v_out [layers, C, N, H_kv, D], status); rows that are absent (lane_nodes),
    of an offending lane or in a page outside the pool keep what k_out and v_out held (zeros if they are not given)."""
    device = R._device(slot_ids, "slot_ids")
    n, arrays = _layers(caches, sh, device, "kv4_read_layers")
    shape = (n, sh.n_seqs, sh.n_nodes, sh.n_kv_heads, sh.head_dim)
    k_out, v_out = (torch.zeros(shape, dtype=sh.dtype, device=device) if t is None else t for t in (k_out, v_out))
    status = R._status_word(status, device)
    R._call(device, _library().gdn_kv4_read_layers, "gdn_kv4_read_layers", ctypes.byref(R._cs(sh)), n, arrays,
            R._ptr(slot_ids, "slot_ids", torch.int32, (sh.n_seqs,), device),
            R._ptr(page_table, "page_table", torch.int32, (sh.n_slots, sh.max_pages), device),
            R._ptr(first_row, "first_row", torch.int32, (sh.n_seqs,), device),
            R._opt(lane_nodes, "lane_nodes", torch.int32, (sh.n_seqs,), device),
            R._ptr(k_out, "k_out", sh.dtype, shape, device), R._ptr(v_out, "v_out", sh.dtype, shape, device), status.data_ptr())
    return k_out, v_out, status
