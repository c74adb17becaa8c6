"""Seeded inputs of the paged-cache and acceptance calls, and comparisons with their tolerances."""

from __future__ import annotations

import numpy as np
import torch

import gated_deltanet_speculative_amd as gdn

SENTINEL = -768.0  # exact in every type
#: half a step of a rounding to the type, relative to the value
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def as_numpy(t: torch.Tensor) -> np.ndarray:
    """The values of a tensor, exactly (16-bit types as float32)."""
    return t.float().cpu().numpy() if t.is_floating_point() and t.dtype != torch.float64 else t.cpu().numpy()


def dev(a, dtype=None) -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def random_parents(rng, C, N, low=-1):
    """Node i hangs on a node in [low, i - 1] (the first on the prefix)."""
    return np.array([[int(rng.integers(low, i)) if i > 0 else -1 for i in range(N)] for _ in range(C)], np.int32)


class Paged:
    """Slots, scattered pages and random caches for C lanes of the given committed lengths."""

    def __init__(self, C, N, Hq, Hkv, D, page, dtype, lens, seed=0, extra_slots=2, spare_pages=2, layers=0):
        rng = np.random.default_rng(seed)
        self.rng, self.C, self.N = rng, C, N
        P = C + extra_slots
        need = [-(-(n + N) // page) for n in lens]
        n_pages, max_pages = sum(need) + spare_pages, max(need)
        self.slots = rng.permutation(P)[:C].astype(np.int32)
        ids = rng.permutation(n_pages)
        self.table = np.full((P, max_pages), -1, np.int32)
        self.len = np.zeros(P, np.int32)
        at = 0
        for c in range(C):
            self.table[self.slots[c], :need[c]] = ids[at:at + need[c]]
            self.len[self.slots[c]] = lens[c]
            at += need[c]
        self.sh = gdn.AttnShape(C, N, P, Hq, Hkv, D, page, n_pages, max_pages, dtype)
        lead = (layers,) if layers else ()
        self.k, self.v = (dev(rng.standard_normal(lead + self.sh.cache_shape).astype(np.float32), dtype) for _ in range(2))

    def places(self):
        return dev(self.slots), dev(self.table), dev(self.len)

    def normal(self, *shape, std=1.0, dtype=None):
        return dev((self.rng.standard_normal(shape) * std).astype(np.float32), dtype or self.sh.dtype)


def attention_tolerance(dtype, D, mag, out, big, rows, gated):
    """Largest error of each output, from the roundings on its way.

    `mag` is sum w |V| / sum w, `big` the largest scale * sum |q||k| of a row.  A score of D products summed in
    32 bits is off by at most D 2^-23 big (2^-23: the matrix unit's own summation need not round to nearest),
    the base-2 exponential and the scaled subtraction by 2^-22 (1 + big) more; both weigh numerator and sum.
    A 16-bit path rounds the weights once (half a step); the sums over `rows` rows add rows 2^-23 twice; joining
    parts multiplies by one more exponential of the same error.  The output is rounded once.  The gate's
    exponential and reciprocal are good to 2^-19 for |z| < 8."""
    half = HALF_STEP[dtype]
    score = D * 2.0 ** -23 * big + 2.0 ** -21 * (1 + big)
    rel = 2 * score + 2 * (rows + 16) * 2.0 ** -23 + (half if dtype != torch.float32 else 0.0) + (2.0 ** -19 if gated else 0.0)
    return mag * rel * (1 + 2.0 ** -6) + half * np.abs(out) * (1 + 2.0 ** -6) + 1e-30


def check_attention(got: torch.Tensor, res: dict, dtype, gated=False, ctx=""):
    """Every computed row against the oracle's; every other row still the sentinel."""
    g = as_numpy(got).astype(np.float64)
    C, N, Hq, D = g.shape
    worst = 0.0
    for c in range(C):
        for i in range(N):
            if (c, i) not in res:
                assert (g[c, i] == SENTINEL).all(), f"{ctx}: row {(c, i)} was written"
                continue
            out, mag, big, rows = res[c, i]
            tol = attention_tolerance(dtype, D, mag, out, big, rows, gated)
            err = np.abs(g[c, i] - out)
            assert np.isfinite(g[c, i]).all(), f"{ctx}: row {(c, i)} is not finite"
            worst = max(worst, float(np.max(err / tol)))
            assert (err <= tol).all(), f"{ctx}: row {(c, i)} off by {err.max()} ({float(np.max(err / tol)):.2f} of the tolerance)"
    return worst
