"""Binding of the gdn_logits.h call: penalties, biases, masks and temperatures between the target's logits and the
acceptance of the draft.

Argument marshalling only: a missing output or workspace is allocated here, the tensors are checked and the call made by the
binding's extension (csrc/marshal.cpp).  There is no fallback.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import _round as R
from ._lib import load_library

STATUS_RULE = 512
LOGITS_EXPORTED = ("gdn_adjust_logits", "gdn_adjust_logits_workspace_size")

_i32, _vp = ctypes.c_int32, ctypes.c_void_p


class _CLogitsShape(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("n_seqs", "n_nodes", "n_slots", "vocab", "max_history", "max_bias", "dtype", "out_dtype")]


class _CLogitRules(ctypes.Structure):
    _fields_ = [(n, _vp) for n in ("history", "history_len", "prompt_len", "repetition", "presence", "frequency", "bias_tokens",
                                   "bias", "temperature")]


class LogitsShape(NamedTuple):
    """Sizes of one call (gdn_logits_shape); dtype is that of the logits, out_dtype that of the result (the same, or
    float32)."""

    n_seqs: int
    n_nodes: int
    n_slots: int
    vocab: int
    max_history: int = 0
    max_bias: int = 0
    dtype: torch.dtype = torch.bfloat16
    out_dtype: torch.dtype = torch.float32

    def c_struct(self) -> _CLogitsShape:
        return _CLogitsShape(*self[:6], R._dtype_code(self.dtype), R._dtype_code(self.out_dtype))


@functools.lru_cache(maxsize=1)
def _library():
    """The library with the prototypes of these calls, for callers through ctypes (the calls below go by their addresses)."""
    lib = load_library()
    sp = ctypes.POINTER(_CLogitsShape)
    lib.gdn_adjust_logits.argtypes = [sp, _vp, ctypes.c_int64, ctypes.POINTER(_CLogitRules)] + [_vp] * 7 + [ctypes.c_size_t, _vp, _vp]
    lib.gdn_adjust_logits.restype = _i32
    lib.gdn_adjust_logits_workspace_size.argtypes = [sp]
    lib.gdn_adjust_logits_workspace_size.restype = ctypes.c_size_t
    return lib


def adjust_logits_workspace_size(sh: LogitsShape) -> int:
    """Bytes of device workspace adjust_logits needs for this shape where there is a temperature (0 for an invalid shape)."""
    return int(_library().gdn_adjust_logits_workspace_size(ctypes.byref(R._shape(sh)[0])))


def adjust_logits(sh: LogitsShape, logits, slot_ids, history=None, history_len=None, prompt_len=None, repetition=None,
                  presence=None, frequency=None, bias_tokens=None, bias=None, mask=None, tokens=None, parents=None,
                  lane_nodes=None, temperature=None, out=None, workspace=None, status=None):
    """A slot's rules on the logits [C, N, V] after every node of a draft: penalties for the tokens of its history
    [P, max_history] (of which history_len [P] entries are in use, the first prompt_len [P] of them the prompt's) and of
    the node's path (`tokens` [C, N], along `parents`, or along the chain), biases (bias_tokens, bias [P, max_bias]) and
    a grammar's mask ([C, N, ceil(V / 32)] int32, a bit for every allowed token).  repetition, presence and
    frequency are float32 [P].  With temperature [P] the result is the probabilities (0: one at the largest), which
    draft_accept takes.  `workspace` is a float32 device tensor of at least adjust_logits_workspace_size(sh) bytes
    (with a temperature; allocated per call when omitted).  Returns (out [C, N, V], status)."""
    device = R._device(logits, "logits")
    call, f = R._call_of("adjust_logits", _library)
    held, shape = R._shape(sh)  # (held: the struct lives through the call)
    if out is None:
        out = torch.empty((sh.n_seqs, sh.n_nodes, sh.vocab), dtype=sh.out_dtype, device=device)
    status = R._status_word(status, device)
    if workspace is None and temperature is not None:
        workspace = torch.empty(max(adjust_logits_workspace_size(sh) // 4, 1), dtype=torch.float32, device=device)
    R._call(device, call, "gdn_adjust_logits", f, shape, device, logits, history, history_len, prompt_len,
            repetition, presence, frequency, bias_tokens, bias, temperature, mask, tokens, parents, lane_nodes, slot_ids, out, workspace,
            status)
    return out, status
