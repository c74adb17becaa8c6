"""Binding of the gdn_kv4.h calls: the attention layers' part of a round over a cache held in 4 bits.

Argument marshalling only: missing outputs are allocated here, the tensors are checked and the calls made by the binding's
extension (csrc/marshal.cpp).  There is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
import math
from typing import NamedTuple

import torch

from . import _round as R
from ._lib import load_library

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


@functools.lru_cache(maxsize=1)
def _library():
    """The library with the prototypes of these calls, for callers through ctypes (the calls below go by their addresses)."""
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
    return lib


def rope_kv4_write(sh: R.AttnShape, q, k, v, inv_freq, cache, slot_ids, page_table, seq_len, positions=None, pair_axis=None,
                   parents=None, lane_nodes=None, q_norm=None, k_norm=None, eps=1e-6, interleaved=False, q_out=None,
                   status=None):
    """Rotary positions of q and k and the write of k and v, quantised to 4 bits, into the slots' pages behind their
    committed rows: rope_kv_write with a Kv4Cache in the place of the two caches.  Returns (q_out, status)."""
    device = R._device(q, "q")
    call, f = R._call_of("rope_kv4_write", _library)
    held, shape = R._shape(sh)  # (held: the struct lives through the call)
    if q_out is None:
        q_out = torch.empty((sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim), dtype=sh.dtype, device=device)
    status = R._status_word(status, device)
    R._call(device, call, "gdn_rope_kv4_write", f, shape, device, q, k, v, inv_freq, cache, slot_ids,
            page_table, seq_len, positions, pair_axis, parents, lane_nodes, q_norm, k_norm, eps, bool(interleaved), q_out, status)
    return q_out, status


def paged_attention_kv4_workspace_size(sh: R.AttnShape) -> int:
    """Bytes of device workspace paged_attention_kv4 needs for this shape (0 for an invalid shape)."""
    return int(_library().gdn_paged_attention_kv4_workspace_size(ctypes.byref(R._shape(sh)[0])))


def paged_attention_kv4(sh: R.AttnShape, q, cache, slot_ids, page_table, seq_len, parents=None, lane_nodes=None, scale=None,
                        gate=None, gate_mode=1, out=None, workspace=None, status=None):
    """Attention of the round's tokens over a 4-bit cache: paged_attention with a Kv4Cache in the place of the two
    caches (`workspace` is at least paged_attention_kv4_workspace_size(sh) bytes).  Returns (out, status)."""
    device = R._device(q, "q")
    call, f = R._call_of("paged_attention_kv4", _library)
    held, shape = R._shape(sh)  # (held: the struct lives through the call)
    if out is None:
        out = torch.empty((sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim), dtype=sh.dtype, device=device)
    status = R._status_word(status, device)
    if workspace is None:
        workspace = torch.empty(max(paged_attention_kv4_workspace_size(sh) // 4, 1), dtype=torch.float32, device=device)
    R._call(device, call, "gdn_paged_attention_kv4", f, shape, device, q, cache, slot_ids, page_table,
            seq_len, parents, lane_nodes, 1.0 / math.sqrt(sh.head_dim) if scale is None else scale, gate, int(gate_mode), out,
            workspace, status)
    return out, status


def kv4_commit_layers(sh: R.AttnShape, caches, slot_ids, page_table, seq_len, accept_node, status, parents=None,
                      lane_nodes=None, new_len=None):
    """Moves the accepted paths' rows of every layer's 4-bit cache together behind the committed rows and returns the
    new lengths [P]: kv_commit_layers with a Kv4Cache of tensors with a leading layer axis, or a sequence of one
    Kv4Cache a layer.  A transaction on the status word: every lane and layer, or nothing."""
    if status is None:
        raise ValueError("kv4_commit_layers needs a status word (the round's transaction flag)")
    device = R._device(status, "status")
    call, f = R._call_of("kv4_commit_layers", _library)
    held, shape = R._shape(sh)  # (held: the struct lives through the call)
    if new_len is None:
        new_len = torch.empty(sh.n_slots, dtype=torch.int32, device=device)
    R._call(device, call, "gdn_kv4_commit_layers", f, shape, device, caches, slot_ids, page_table,
            seq_len, parents, lane_nodes, accept_node, new_len, status)
    return new_len


def _layers(caches) -> int:
    """The layers of a Kv4Cache with a leading layer axis, or of a sequence of one a layer; 1 for what the call refuses."""
    if isinstance(caches, tuple) and len(caches) == 4 and not isinstance(caches[0], tuple):
        k = caches[0]
        return k.shape[0] if isinstance(k, torch.Tensor) and k.dim() == 5 else 1
    return len(caches) if hasattr(caches, "__len__") else 1


def kv4_read_layers(sh: R.AttnShape, caches, slot_ids, page_table, first_row, lane_nodes=None, k_out=None, v_out=None,
                    status=None):
    """Rows first_row[c] .. first_row[c] + N - 1 of every lane's slot as values of sh.dtype, for every layer (caches as in
    kv4_commit_layers).  Returns (k_out, v_out [layers, C, N, H_kv, D], status); rows that are absent (lane_nodes),
    of an offending lane or in a page outside the pool keep what k_out and v_out held (zeros if they are not given)."""
    device = R._device(slot_ids, "slot_ids")
    call, f = R._call_of("kv4_read_layers", _library)
    held, shape = R._shape(sh)  # (held: the struct lives through the call)
    if k_out is None or v_out is None:
        rows = (_layers(caches), sh.n_seqs, sh.n_nodes, sh.n_kv_heads, sh.head_dim)
        k_out, v_out = (torch.zeros(rows, dtype=sh.dtype, device=device) if t is None else t for t in (k_out, v_out))
    status = R._status_word(status, device)
    R._call(device, call, "gdn_kv4_read_layers", f, shape, device, caches, slot_ids, page_table, first_row,
            lane_nodes, k_out, v_out, status)
    return k_out, v_out, status
