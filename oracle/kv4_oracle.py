"""fp64 oracle of the calls in gdn_kv4.h: the 4-bit form by its definition, one block at a time where it is quantised,
around the oracle of the calls over caches of values.  It shares nothing with the HIP path."""

from __future__ import annotations

import math

import numpy as np

from . import round_oracle as R

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BLOCK, LOWEST = 32, -125


def values(codes, scales):
    """float64 values of uint8 codes [..., D / 2] and scales [..., D / 32]."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    x = np.array(MAGNITUDES + tuple(-m for m in MAGNITUDES))[n]
    power = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return x * np.repeat(power, BLOCK, -1)


def exponent(a, most):
    """e of a block whose largest magnitude is a."""
    if a == 0:
        return LOWEST
    m, p = math.frexp(a)  # a = 2m 2^(p - 1), 2m in [1, 2)
    return min(max((p if 2 * m >= 1.75 else p - 1) - 2, LOWEST), most)


def nearest(y):
    """Code of the magnitude nearest to y >= 0, ties to the one of even code, at most 6."""
    best = min(range(8), key=lambda c: (abs(MAGNITUDES[c] - y), c % 2))
    return 7 if y > 6 else best


def quantise(row, float16=False):
    """(codes, scales) of a row of D values."""
    row = np.asarray(row, np.float64)
    codes, scales = np.zeros(len(row), np.uint8), np.zeros(len(row) // BLOCK, np.uint8)
    for b in range(len(scales)):
        x = row[BLOCK * b:BLOCK * (b + 1)]
        if not np.isfinite(x).all():
            scales[b] = 255
            continue
        e = exponent(float(np.abs(x).max()), 13 if float16 else 125)
        scales[b] = e + 127
        for j, v in enumerate(x):
            codes[BLOCK * b + j] = nearest(abs(v) / 2.0 ** e) + (8 if math.copysign(1.0, v) < 0 else 0)
    return codes[0::2] | codes[1::2] << 4, scales


def rope_rows(q, k, v, inv_freq, heads, page, n_pages, *where, **kw):
    """q rows, {(slot, row): (k, v)} unquantised rows that the call writes, and the status."""
    slots, table, length = where
    nan = np.full((n_pages, heads, page, k.shape[-1]), np.nan)
    kc, vc = nan.copy(), nan.copy()
    rows, status = R.rope_kv_write(q, k, v, inv_freq, kc, vc, slots, table, length, **kw)
    return rows, kc, vc, status


def read(codes, scales, slots, table, first, N, nodes=None):
    """({(c, i): values [Hkv, D]}, status) of one layer's array."""
    n_pages, _, page, _ = codes.shape
    out, status = {}, 0
    for c, s in enumerate(slots):
        n = N if nodes is None else int(nodes[c])
        if s == -1:
            continue
        bits = 0
        if not 0 <= n <= N:
            bits |= R.NODES
        if s < -1 or s >= len(table):
            bits |= R.SLOT_RANGE
        if first[c] < 0 or int(first[c]) + max(n, 0) > table.shape[1] * page:
            bits |= R.LENGTH
        status |= bits
        for i in range(0 if bits else n):
            pid, at = int(table[s, (int(first[c]) + i) // page]), (int(first[c]) + i) % page
            if 0 <= pid < n_pages:
                out[c, i] = values(codes[pid, :, at], scales[pid, :, at])
            else:
                status |= R.PAGE
    return out, status
