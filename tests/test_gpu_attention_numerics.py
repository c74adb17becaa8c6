"""Attention over the paged cache where its arithmetic is strained, in every kernel: weights many powers of two
below the largest one, rows without anything to attend to behind a gate, scores of any size."""

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gpu_util import log
from oracle import round_oracle as R
from round_util import SENTINEL, Paged, as_numpy, attention_tolerance, dev

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
# Head layouts that reach every kernel with 8 nodes: few rows, 64, 128 and 256 rows a workgroup, pairs of waves, each type
KERNELS = [(64, 2), (64, 8), (64, 16), (64, 40), (128, 2), (128, 8), (128, 16), (128, 40), (256, 1), (256, 2), (256, 40)]


def _rows(pg, c, n):
    """(page, place) of the first n rows of lane c's cache."""
    t = np.arange(n)
    return pg.table[pg.slots[c], t // pg.sh.page_size].astype(np.int64), t % pg.sh.page_size


def _attend(pg, q, **kw):
    out = torch.full(tuple(q.shape), SENTINEL, dtype=pg.sh.dtype, device="cuda")
    table = kw.pop("table", pg.table)
    ws = torch.full((max(gdn.paged_attention_workspace_size(pg.sh) // 4, 1),), float("nan"), device="cuda")
    _, status = gdn.paged_attention(pg.sh, q, pg.k, pg.v, dev(pg.slots), dev(table), dev(pg.len), out=out, workspace=ws, **kw)
    torch.cuda.synchronize()
    return out, int(status.item())


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
def test_small_weights_beside_a_large_one(dtype, D, G):
    """Every 64th row outscores the others, which are equal, by 18 to 24 powers of two and has a value of zero: the
    output is what the small weights leave, and their rounding is the same for all of them.

    In float16 a weight below 2^-14 is off by up to 2^-25.  The largest weight of a row, and so the sum, is at least
    2^9, the exponentials' base lying 9 powers of two below a running maximum: each row adds up to 2^-34 |v|."""
    C, N, lens = 2, 8, [1000, 700]
    pg = Paged(C, N, G, 1, D, 48, dtype, lens, seed=D + G)
    k, v = as_numpy(pg.k), np.empty(pg.sh.cache_shape, np.float32)
    v[:] = pg.rng.uniform(1.0, 2.0, v.shape)
    k[..., 0] = 0.0
    for c in range(C):
        pid, at = _rows(pg, c, lens[c])
        k[pid[::64], 0, at[::64], 0] = 16.0
        v[pid[::64], 0, at[::64]] = 0.0
    pg.k, pg.v = dev(k, dtype), dev(v, dtype)
    q = np.zeros((C, N, G, D), np.float32)
    q[..., 0] = pg.rng.integers(48, 65, (C, N, G)) / 64.0
    q = dev(q, dtype)
    scale = 24.0 / (16.0 * 1.4426950408889634)
    log(f"[attn small weights] {dtype} D={D} G={G}")
    out, status = _attend(pg, q, scale=scale)
    res, bits = R.paged_attention(as_numpy(q), as_numpy(pg.k), as_numpy(pg.v), pg.slots, pg.table, pg.len, scale=scale)
    assert status == bits == 0
    got = as_numpy(out).astype(np.float64)
    for (c, i), (want, mag, big, rows) in res.items():
        tol = attention_tolerance(dtype, D, mag, want, big, rows, False) + (rows * 2.0 ** -34 * 2.0 if dtype == HF else 0.0)
        err = np.abs(got[c, i] - want)
        assert (err <= tol).all(), f"row {(c, i)}: {float(np.max(err / tol)):.2f} of the tolerance, {float(np.max(err / want)):.2e} relative"


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
@pytest.mark.parametrize("mode", [0, 1])
def test_rows_without_anything_attended_are_zero_behind_any_gate(dtype, D, G, mode):
    """No page in the pool, or every score minus infinity: zeros, whatever the gate holds."""
    C, N = 2, 8
    pg = Paged(C, N, G, 1, D, 48, dtype, [700, 3], seed=D + G)
    q = dev(pg.rng.uniform(0.5, 1.0, (C, N, G, D)).astype(np.float32), dtype)
    gate = torch.tensor([float("nan"), float("inf"), -float("inf"), 1.0], device="cuda").to(dtype).repeat(C, N, G, D // 4)
    log(f"[attn gate of nothing] {dtype} D={D} G={G} mode={mode}")
    out, status = _attend(pg, q, gate=gate, gate_mode=mode, table=np.full_like(pg.table, -1))
    assert status == R.PAGE and (as_numpy(out) == 0).all()
    pg.k.fill_(-float("inf"))
    out, status = _attend(pg, q, gate=gate, gate_mode=mode)
    assert status == 0 and (as_numpy(out) == 0).all()


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(dtype, D, G, sign):
    """Scores of 2^33 and more, far apart: the row of the largest one weighs 1, every other one nothing, so the output
    is its value, exactly."""
    C, N, lens = 2, 8, [500, 130]
    pg = Paged(C, N, G, 1, D, 48, dtype, lens, seed=D + G)
    k = as_numpy(pg.k)
    size = np.zeros((C, max(lens) + N))
    for c in range(C):
        n = lens[c] + N
        # distinct values: consecutive float16 ones from 16 on (a 2^-11th apart), bfloat16 ones from 1 on (a 2^-8th)
        order = pg.rng.permutation(n)
        bits = (0x4C00 if dtype == HF else 0x3F80) + order.astype(np.uint16)
        size[c, :n] = sign * (bits.view(np.float16) if dtype == HF else (bits.astype(np.uint32) << 16).view(np.float32))
        pid, at = _rows(pg, c, n)
        k[pid, 0, at, 0] = size[c, :n]
    pg.k = dev(k, dtype)
    q = np.zeros((C, N, G, D), np.float32)
    q[..., 0] = np.where(np.arange(G) % 2 == 0, 1.0, 0.75) * (60000.0 if dtype == HF else 1e18)
    log(f"[attn large scores] {dtype} D={D} G={G} sign={sign}")
    out, status = _attend(pg, dev(q, dtype), scale=8192.0 if dtype == HF else 0.3)
    assert status == 0
    got, v = as_numpy(out), as_numpy(pg.v)
    for c in range(C):
        for i in range(N):
            best = int(np.argmax(size[c, :lens[c] + i + 1]))
            pid, at = _rows(pg, c, best + 1)
            assert np.array_equal(got[c, i], np.broadcast_to(v[pid[-1], 0, at[-1]], (G, D))), f"row {(c, i)}: {got[c, i, 0, :4]}"


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
def test_equal_scores_of_any_size(dtype, D, G):
    """Keys that are all the same: the mean of the attended values, at scores of 2^10 to 2^37 of either sign (some rows of a
    wave beyond the size at which its scores become differences, others not)."""
    C, N, lens = 2, 8, [500, 130]
    pg = Paged(C, N, G, 1, D, 48, dtype, lens, seed=D + G)
    k = as_numpy(pg.k)
    k[..., 0] = 16.0
    pg.k = dev(k, dtype)
    q = np.zeros((C, N, G, D), np.float32)
    q[..., 0] = pg.rng.choice([-1, 1], (C, N, G)) * 2.0 ** pg.rng.integers(-6, 7, (C, N, G)) * pg.rng.integers(128, 256, (C, N, G)) / 128
    q = dev(q, dtype)
    res, _ = R.paged_attention(np.zeros_like(as_numpy(q)), k, as_numpy(pg.v), pg.slots, pg.table, pg.len)
    for scale in (2.0 ** 12, 2.0 ** 15, 3.0 * 2.0 ** 18, 1.7 * 2.0 ** 24):
        out, status = _attend(pg, q, scale=scale)
        assert status == 0
        got = as_numpy(out).astype(np.float64)
        for (c, i), (want, mag, _, rows) in res.items():
            tol = attention_tolerance(dtype, D, mag, want, 0.0, rows, False)
            err = np.abs(got[c, i] - want)
            assert (err <= tol).all(), f"scale {scale}, row {(c, i)}: {float(np.max(err / tol)):.2f} of the tolerance"


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
def test_infinite_values_of_committed_rows(dtype, D, G):
    """An infinity in a row that every node attends to, in a tile without a mask, reaches every node in its column."""
    C, N, lens = 2, 8, [500, 300]
    pg = Paged(C, N, G, 1, D, 48, dtype, lens, seed=D + G)
    q = pg.normal(C, N, G, D)
    clean = as_numpy(_attend(pg, q)[0])
    for c in range(C):
        pid, at = _rows(pg, c, lens[c])
        pg.v[int(pid[200]), 0, int(at[200]), 7] = float("inf")
        pg.v[int(pid[1]), 0, int(at[1]), D - 1] = -float("inf")
        pg.v[int(pid[90]), 0, int(at[90]), 30] = float("nan")
    got = as_numpy(_attend(pg, q)[0]).copy()
    assert np.isposinf(got[..., 7]).all() and np.isneginf(got[..., D - 1]).all() and np.isnan(got[..., 30]).all()
    for col in (7, D - 1, 30):
        got[..., col] = clean[..., col]
    assert np.array_equal(got, clean)
