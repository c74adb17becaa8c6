"""ctypes binding of the gdn_round.h calls: the attention layers' part of a round and the acceptance.

Argument marshalling only, as in the binding of the recurrence calls: tensors' types, shapes,
devices and layouts are checked, missing outputs allocated, raw pointers and torch's current
stream passed on.  There is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
import math
import struct
from typing import NamedTuple, Optional

import torch

from ._lib import GDN_OK, MAX_LAYERS, GdnError, load_library

STATUS_LENGTH, STATUS_PAGE, STATUS_TOKEN, STATUS_AXIS = 32, 64, 128, 256
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
ROUND_EXPORTED = ("gdn_rope_kv_write", "gdn_paged_attention", "gdn_paged_attention_workspace_size",
                  "gdn_draft_accept", "gdn_draft_accept_workspace_size", "gdn_kv_commit_layers")

_i32, _vp = ctypes.c_int32, ctypes.c_void_p


class _CAttnShape(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("n_seqs", "n_nodes", "n_slots", "n_q_heads", "n_kv_heads", "head_dim", "page_size",
                                    "n_pages", "max_pages", "dtype")]


class _CAcceptShape(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("n_seqs", "n_nodes", "vocab", "dtype")]


class _CRope(ctypes.Structure):
    _fields_ = [("inv_freq", _vp), ("positions", _vp), ("pair_axis", _vp), ("n_axes", _i32), ("rot_dim", _i32),
                ("interleaved", _i32), ("q_norm", _vp), ("k_norm", _vp), ("eps", ctypes.c_float)]


class AttnShape(NamedTuple):
    """Sizes of one attention layer's call (gdn_attn_shape); dtype is a torch dtype."""

    n_seqs: int
    n_nodes: int
    n_slots: int
    n_q_heads: int
    n_kv_heads: int
    head_dim: int
    page_size: int
    n_pages: int
    max_pages: int
    dtype: torch.dtype = torch.bfloat16

    @property
    def cache_shape(self) -> tuple:
        return (self.n_pages, self.n_kv_heads, self.page_size, self.head_dim)

    def c_struct(self) -> _CAttnShape:
        return _CAttnShape(*self[:9], _dtype_code(self.dtype))


class AcceptShape(NamedTuple):
    """Sizes of one acceptance call (gdn_accept_shape); dtype is that of the probabilities."""

    n_seqs: int
    n_nodes: int
    vocab: int
    dtype: torch.dtype = torch.float32

    def c_struct(self) -> _CAcceptShape:
        return _CAcceptShape(*self[:3], _dtype_code(self.dtype))


def _dtype_code(dtype: torch.dtype) -> int:
    code = DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be one of {', '.join(str(d) for d in DTYPES)}, got {dtype}")
    return code


_calls = None


def _library():
    """The library with the prototypes of these calls (looked up once)."""
    global _calls
    if _calls is None:
        lib = load_library()
        sp, ap = ctypes.POINTER(_CAttnShape), ctypes.POINTER(_CAcceptShape)
        lib.gdn_rope_kv_write.argtypes = [sp, _i32, _vp, _vp, _vp, ctypes.POINTER(_CRope)] + [_vp] * 10
        lib.gdn_paged_attention.argtypes = [sp] + [_vp] * 8 + [ctypes.c_float, _vp, _i32, _vp, _vp, ctypes.c_size_t, _vp, _vp]
        lib.gdn_paged_attention_workspace_size.argtypes = [sp]
        lib.gdn_draft_accept.argtypes = [ap] + [_vp] * 13 + [ctypes.c_size_t, _vp, _vp]
        lib.gdn_draft_accept_workspace_size.argtypes = [ap]
        lib.gdn_kv_commit_layers.argtypes = [sp, _i32] + [_vp] * 11
        for f in ("gdn_rope_kv_write", "gdn_paged_attention", "gdn_draft_accept", "gdn_kv_commit_layers"):
            getattr(lib, f).restype = _i32
        for f in ("gdn_paged_attention_workspace_size", "gdn_draft_accept_workspace_size"):
            getattr(lib, f).restype = ctypes.c_size_t
        _calls = lib
    return _calls


# ---------------------------------------------------------------- marshalling helpers
# A small call is bound by this file, so the tensors' checks are native (csrc/marshal.cpp): _ptr, _opt and _view are
# the extension's functions from the first call on.
def _ptr(*args):
    """Pointer of a contiguous tensor: (tensor, name, dtype, shape, device index)."""
    _load_marshal()
    return _ptr(*args)


def _opt(*args):
    """The same, or None for None."""
    _load_marshal()
    return _opt(*args)


def _view(*args):
    """A gdn_heads_view, as bytes, of a [C, N, heads, D] tensor whose last dimension is contiguous and whose tokens
    are evenly strided over the lanes (a slice of a stacked projection, or a contiguous tensor)."""
    _load_marshal()
    return _view(*args)


def _load_marshal() -> None:
    global _ptr, _opt, _view
    try:
        from . import _marshal
    except ImportError as e:
        raise RuntimeError("_marshal.so is missing: build it with `python -m gated_deltanet_speculative_amd.build`") from e
    _marshal.init(_refuse)
    _ptr, _opt, _view = _marshal.ptr, _marshal.opt, _marshal.view


def _refuse(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if t.device.index != device:
        raise ValueError(f"{name} is on {t.device}, the call's first tensor on cuda:{device}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _device(t, name) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    return t.get_device()


def _status_word(status, device) -> torch.Tensor:
    if status is None:
        return torch.zeros(1, dtype=torch.int32, device=device)
    _ptr(status, "status", torch.int32, (1,), device)
    return status


def _call(device: int, f, name, *args) -> None:
    """f(*args, stream) with torch's current stream of the tensors' device, which is made current: a launch
    goes to the stream's device."""
    if torch._C._cuda_getDevice() == device:
        code = f(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            code = f(*args, torch._C._cuda_getCurrentRawStream(device))
    if code != GDN_OK:
        raise GdnError(code, name)


@functools.lru_cache(maxsize=256)
def _cs(sh):
    """The C struct of a shape (never written to)."""
    return sh.c_struct()


def _places(sh: AttnShape, slot_ids, page_table, seq_len, device) -> tuple:
    return (_ptr(slot_ids, "slot_ids", torch.int32, (sh.n_seqs,), device),
            _ptr(page_table, "page_table", torch.int32, (sh.n_slots, sh.max_pages), device),
            _ptr(seq_len, "seq_len", torch.int32, (sh.n_slots,), device))


def _tree(sh, parents, lane_nodes, device) -> tuple:
    return (_opt(parents, "parents", torch.int32, (sh.n_seqs, sh.n_nodes), device),
            _opt(lane_nodes, "lane_nodes", torch.int32, (sh.n_seqs,), device))


# ---------------------------------------------------------------- the calls
def rope_kv_write(sh: AttnShape, q, k, v, inv_freq, k_cache, v_cache, slot_ids, page_table, seq_len, positions=None,
                  pair_axis=None, parents=None, lane_nodes=None, q_norm=None, k_norm=None, eps=1e-6, interleaved=False,
                  q_out=None, status=None):
    """Rotary positions of q and k (after an optional RMS norm) and the write of k and v into the slots' pages
    behind their committed rows.

    q, k, v are [C, N, heads, D] views (e.g. of the stacked projection) of sh.dtype or float32; inv_freq is a
    float64 device tensor of rot_dim / 2 entries.  positions is [C, N, n_axes] int32 (default: the committed
    length plus the node's depth) and pair_axis [rot_dim / 2] int32 names each pair's axis (default 0); q_norm,
    k_norm are float32 [D].  Returns (q_out [C, N, H_q, D], status).
    """
    device = _device(q, "q")
    C, N, D = sh.n_seqs, sh.n_nodes, sh.head_dim
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a one-dimensional float64 tensor of rot_dim / 2 entries")
    half = inv_freq.shape[0]
    n_axes = 1
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dim() != 3:
            raise ValueError("positions must be a [C, N, n_axes] int32 tensor")
        n_axes = positions.shape[2]
    if q_out is None:
        q_out = torch.empty((C, N, sh.n_q_heads, D), dtype=sh.dtype, device=device)
    status = _status_word(status, device)
    x = torch.float32 if q.dtype is torch.float32 else sh.dtype
    q_shape, kv_shape = (C, N, sh.n_q_heads, D), (C, N, sh.n_kv_heads, D)
    rope = _CRope(_ptr(inv_freq, "inv_freq", torch.float64, (half,), device),
                  _opt(positions, "positions", torch.int32, (C, N, n_axes), device),
                  _opt(pair_axis, "pair_axis", torch.int32, (half,), device), n_axes, 2 * half, int(bool(interleaved)),
                  _opt(q_norm, "q_norm", torch.float32, (D,), device),
                  _opt(k_norm, "k_norm", torch.float32, (D,), device), eps)
    _call(device, _library().gdn_rope_kv_write, "gdn_rope_kv_write", ctypes.byref(_cs(sh)), _dtype_code(x),
          _view(q, "q", x, q_shape, device), _view(k, "k", x, kv_shape, device), _view(v, "v", x, kv_shape, device),
          ctypes.byref(rope), _ptr(k_cache, "k_cache", sh.dtype, sh.cache_shape, device),
          _ptr(v_cache, "v_cache", sh.dtype, sh.cache_shape, device), *_places(sh, slot_ids, page_table, seq_len, device),
          *_tree(sh, parents, lane_nodes, device),
          _ptr(q_out, "q_out", sh.dtype, q_shape, device), status.data_ptr())
    return q_out, status


def paged_attention_workspace_size(sh: AttnShape) -> int:
    """Bytes of device workspace paged_attention needs for this shape (0 for an invalid shape)."""
    return int(_library().gdn_paged_attention_workspace_size(ctypes.byref(_cs(sh))))


def paged_attention(sh: AttnShape, q, k_cache, v_cache, slot_ids, page_table, seq_len, parents=None, lane_nodes=None,
                    scale=None, gate=None, gate_mode=1, out=None, workspace=None, status=None):
    """Attention of the round's tokens (their rows already in the caches) over the committed rows and over their
    own ancestors: along `parents` [C, N], or along the chain.  scale defaults to 1 / sqrt(D).  With gate (a
    [C, N, H_q, D] view) the output is multiplied by silu(gate) (gate_mode 0) or sigmoid(gate) (1).  `workspace`
    is a float32 device tensor of at least paged_attention_workspace_size(sh) bytes (allocated per call when
    omitted).  Returns (out [C, N, H_q, D], status)."""
    device = _device(q, "q")
    shape = (sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim)
    if out is None:
        out = torch.empty(shape, dtype=sh.dtype, device=device)
    status = _status_word(status, device)
    lib, cs = _library(), ctypes.byref(_cs(sh))
    if workspace is None:
        workspace = torch.empty(max(lib.gdn_paged_attention_workspace_size(cs) // 4, 1), dtype=torch.float32, device=device)
    else:
        workspace = _scratch(workspace, device)
    _call(device, lib.gdn_paged_attention, "gdn_paged_attention", cs, _ptr(q, "q", sh.dtype, shape, device),
          _ptr(k_cache, "k_cache", sh.dtype, sh.cache_shape, device),
          _ptr(v_cache, "v_cache", sh.dtype, sh.cache_shape, device), *_places(sh, slot_ids, page_table, seq_len, device),
          *_tree(sh, parents, lane_nodes, device), 1.0 / math.sqrt(sh.head_dim) if scale is None else scale,
          None if gate is None else _view(gate, "gate", sh.dtype, shape, device), int(gate_mode),
          _ptr(out, "out", sh.dtype, shape, device), workspace.data_ptr(), workspace.numel() * 4, status.data_ptr())
    return out, status


def _scratch(workspace, device) -> torch.Tensor:
    if not (isinstance(workspace, torch.Tensor) and workspace.dtype is torch.float32 and workspace.get_device() == device
            and workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous float32 tensor on the call's device")
    return workspace


def draft_accept_workspace_size(sh: AcceptShape) -> int:
    """Bytes of device workspace draft_accept needs for this shape (0 for an invalid shape)."""
    return int(_library().gdn_draft_accept_workspace_size(ctypes.byref(_cs(sh))))


def draft_accept(sh: AcceptShape, target, tokens, root_target=None, draft=None, parents=None, lane_nodes=None,
                 slot_ids=None, u_accept=None, u_next=None, accept_node=None, n_accept=None, next_token=None,
                 workspace=None, status=None):
    """Tests the drafted tokens [C, N] against the target's probabilities: target [C, N, V] after each node and
    root_target [C, V] after the committed prefix (without it the lowest child of the prefix is a token already
    drawn).  draft [C, N, V] is the distribution each node's token was drawn from (chains only; without it the
    nodes are candidates).  u_accept [C, N] and u_next [C] are the random numbers; without them the walk is
    greedy.  Returns (accept_node, n_accept, next_token, status); accept_node is what the commits take."""
    device = _device(target, "target")
    C, N, V = sh.n_seqs, sh.n_nodes, sh.vocab
    outs = []
    for t, name in ((accept_node, "accept_node"), (n_accept, "n_accept"), (next_token, "next_token")):
        if t is None:
            t = torch.full((C,), -1, dtype=torch.int32, device=device)
        _ptr(t, name, torch.int32, (C,), device)
        outs.append(t)
    status = _status_word(status, device)
    lib, cs = _library(), ctypes.byref(_cs(sh))
    if workspace is None:
        workspace = torch.empty(max(lib.gdn_draft_accept_workspace_size(cs) // 4, 1), dtype=torch.float32, device=device)
    else:
        workspace = _scratch(workspace, device)
    _call(device, lib.gdn_draft_accept, "gdn_draft_accept", cs, _ptr(target, "target", sh.dtype, (C, N, V), device),
          _opt(root_target, "root_target", sh.dtype, (C, V), device), _opt(draft, "draft", sh.dtype, (C, N, V), device),
          _ptr(tokens, "tokens", torch.int32, (C, N), device), *_tree(sh, parents, lane_nodes, device),
          _opt(slot_ids, "slot_ids", torch.int32, (C,), device), _opt(u_accept, "u_accept", torch.float32, (C, N), device),
          _opt(u_next, "u_next", torch.float32, (C,), device), *(t.data_ptr() for t in outs), workspace.data_ptr(),
          workspace.numel() * 4, status.data_ptr())
    return (*outs, status)


def _layer_pointers(caches, name: str, sh: AttnShape, device) -> list:
    """Pointers of the layers' caches: a sequence of tensors, or one contiguous tensor with a leading layer axis."""
    if isinstance(caches, torch.Tensor):
        p = _ptr(caches, name, sh.dtype, (caches.shape[0] if caches.dim() else 0, *sh.cache_shape), device)
        step = caches.element_size() * math.prod(sh.cache_shape)
        return [p + i * step for i in range(caches.shape[0])]
    return [_ptr(t, f"{name}[{i}]", sh.dtype, sh.cache_shape, device) for i, t in enumerate(caches)]


def kv_commit_layers(sh: AttnShape, k_caches, v_caches, slot_ids, page_table, seq_len, accept_node, status, parents=None,
                     lane_nodes=None, new_len=None):
    """Moves the accepted paths' rows of every layer's caches together behind the committed rows and returns the
    new lengths [P] (seq_len of the next round).  k_caches and v_caches are sequences of one tensor per layer, or one
    tensor each with a leading layer axis.  A transaction on the status word: every lane and layer, or nothing."""
    if status is None:
        raise ValueError("kv_commit_layers needs a status word (the round's transaction flag)")
    device = _device(status, "status")
    if new_len is None:
        new_len = torch.empty(sh.n_slots, dtype=torch.int32, device=device)
    ks, vs = (_layer_pointers(t, n, sh, device) for t, n in ((k_caches, "k_caches"), (v_caches, "v_caches")))
    if len(ks) != len(vs):
        raise ValueError("kv_commit_layers: k_caches and v_caches differ in length")
    if not 1 <= len(ks) <= MAX_LAYERS:
        raise ValueError(f"kv_commit_layers: {len(ks)} layers, expected 1..{MAX_LAYERS}")
    arr = struct.Struct(f"{len(ks)}P").pack
    _call(device, _library().gdn_kv_commit_layers, "gdn_kv_commit_layers", ctypes.byref(_cs(sh)), len(ks), arr(*ks),
          arr(*vs), *_places(sh, slot_ids, page_table, seq_len, device), *_tree(sh, parents, lane_nodes, device),
          _ptr(accept_node, "accept_node", torch.int32, (sh.n_seqs,), device),
          _ptr(new_len, "new_len", torch.int32, (sh.n_slots,), device),
          _ptr(status, "status", torch.int32, (1,), device))
    return new_len
