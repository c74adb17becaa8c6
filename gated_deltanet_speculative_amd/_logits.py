"""ctypes binding of the gdn_logits.h call: penalties, biases, masks and temperatures between the target's logits and the
acceptance of the draft.

Argument marshalling only, as in the binding of the gdn_round.h calls, whose helpers it uses.  There is no fallback.
"""

from __future__ import annotations

import ctypes
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


_calls = None


def _library():
    """The library with the prototypes of these calls (looked up once)."""
    global _calls
    if _calls is None:
        lib = load_library()
        sp = ctypes.POINTER(_CLogitsShape)
        lib.gdn_adjust_logits.argtypes = [sp, _vp, ctypes.c_int64, ctypes.POINTER(_CLogitRules)] + [_vp] * 7 + [ctypes.c_size_t, _vp, _vp]
        lib.gdn_adjust_logits.restype = _i32
        lib.gdn_adjust_logits_workspace_size.argtypes = [sp]
        lib.gdn_adjust_logits_workspace_size.restype = ctypes.c_size_t
        _calls = lib
    return _calls


def adjust_logits_workspace_size(sh: LogitsShape) -> int:
    """Bytes of device workspace adjust_logits needs for this shape where there is a temperature (0 for an invalid shape)."""
    return int(_library().gdn_adjust_logits_workspace_size(ctypes.byref(R._cs(sh))))


def _rows(logits, sh, device) -> tuple:
    """Address and row stride of [C, N, V] logits whose rows are contiguous and evenly strided (a slice of a padded
    vocabulary, or a contiguous tensor)."""
    shape = (sh.n_seqs, sh.n_nodes, sh.vocab)
    if logits.dtype != sh.dtype or tuple(logits.shape) != shape or logits.get_device() != device or logits.layout != torch.strided:
        R._refuse(logits, "logits", sh.dtype, shape, device)
    C, N, V = shape
    step = logits.stride(1) if N > 1 else logits.stride(0) if C > 1 else V
    if (V > 1 and logits.stride(2) != 1) or (N > 1 and C > 1 and logits.stride(0) != N * step):
        raise ValueError("logits: the values of a row must be contiguous and the rows evenly strided")
    return logits.data_ptr(), step


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
    C, N, P, V = sh[:4]
    if out is None:
        out = torch.empty((C, N, V), dtype=sh.out_dtype, device=device)
    status = R._status_word(status, device)
    lib, cs = _library(), ctypes.byref(R._cs(sh))
    if workspace is not None:
        workspace = R._scratch(workspace, device)
    elif temperature is not None:
        workspace = torch.empty(max(lib.gdn_adjust_logits_workspace_size(cs) // 4, 1), dtype=torch.float32, device=device)
    slot = lambda t, name, dtype=torch.float32: R._opt(t, name, dtype, (P,), device)  # noqa: E731
    i32, f32 = torch.int32, torch.float32
    rules = _CLogitRules(R._opt(history, "history", i32, (P, sh.max_history), device), slot(history_len, "history_len", i32),
                         slot(prompt_len, "prompt_len", i32), slot(repetition, "repetition"), slot(presence, "presence"),
                         slot(frequency, "frequency"), R._opt(bias_tokens, "bias_tokens", i32, (P, sh.max_bias), device),
                         R._opt(bias, "bias", f32, (P, sh.max_bias), device), slot(temperature, "temperature"))
    R._call(device, lib.gdn_adjust_logits, "gdn_adjust_logits", cs, *_rows(logits, sh, device), ctypes.byref(rules),
            R._opt(mask, "mask", i32, (C, N, (V + 31) // 32), device), R._opt(tokens, "tokens", i32, (C, N), device),
            *R._tree(sh, parents, lane_nodes, device), R._ptr(slot_ids, "slot_ids", i32, (C,), device),
            R._ptr(out, "out", sh.out_dtype, (C, N, V), device), None if workspace is None else workspace.data_ptr(),
            0 if workspace is None else workspace.numel() * 4, status.data_ptr())
    return out, status
