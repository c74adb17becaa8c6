"""Edges of the logits' rules on the GPU against the fp64 oracle: temperatures that are no normal numbers; long
lists of biases with tokens that occur twice; every value of rows with infinities, NaN and the type's lowest value; the
rounding of a repetition."""

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gpu_util import log
from oracle import logits_oracle as L
from round_util import as_numpy, dev
from test_gpu_logits import BF, FP, HF, Call, expected

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [50, 9001])
@pytest.mark.parametrize("temp", [2.0 ** -149, 2.0 ** -140, 1e-39, 2.0 ** -127, 2.0 ** -126, 2.0 ** -125])
def test_temperatures_below_the_normal_numbers(temp, V):
    """Logits of a few of these temperatures' sizes, and among them ones of ordinary size and of the type's range.

    Every small logit is a multiple of 2^-149 and fits 24 bits with its neighbours, so differences are exact; halves of them
    are off by 2^-150 each, two of which come to 2^-22 of an exponent of e at T = 2^-126 (below, nothing is halved).  The
    exponent has the roundings of a quotient (or factor), of log2(e) and of a product: 2^-22 of itself; the exponential
    2^-22; the sum and the reciprocal as in `expected`.  Exponentials below 2^-126 may be flushed."""
    call = Call(2, 3, V, FP, FP, history=0, bias=0, mask=False, tokens=False, seed=21)
    temp = float(np.float32(temp))
    steps = max(1, int(temp / 2.0 ** -149 / 8))
    x = call.rng.integers(-20, 1, (2, 3, V)).astype(np.float64) * steps * 2.0 ** -149
    x[:, 0, ::7] = -1.0
    x[:, 1, 3], x[:, 1, 11] = -3e38, -np.inf
    x[0, 2, 5] = 3e38  # (one alone at the top: all others are nothing beside it)
    call.logits = dev(x.astype(np.float32))
    call.rules = dict(P=call.sh.n_slots, temperature=np.full(call.sh.n_slots, temp, np.float32))
    got, status = call.run()
    g, x, worst = as_numpy(got).astype(np.float64), as_numpy(call.logits).astype(np.float64), 0.0
    assert status == 0
    for c in range(2):
        for i in range(3):
            want = L.probabilities(x[c, i], temp)
            arg = np.where(want > 0, 2.0 ** -22 * np.abs((x[c, i] - x[c, i].max()) / temp), 0.0) + 2.0 ** -22
            tol = want * (arg + (want * arg).sum() + 2.0 ** -22 + 80 * 2.0 ** -23) * (1 + 2.0 ** -6) + 1e-35
            worst = max(worst, float((np.abs(g[c, i] - want) / tol).max()))
    log(f"[logits] T={temp:.1e} V={V}: worst error {worst:.3f} of the tolerance")
    assert worst <= 1 and g[0, 2, 5] == 1


@pytest.mark.parametrize("kind", ["one", "pairs", "equal", "zeros"])
@pytest.mark.parametrize("B", [3, 513, 1024])
@pytest.mark.parametrize("temp", [False, True])
def test_long_bias_lists_with_tokens_that_occur_twice(B, kind, temp):
    """The sums bit for bit: float32 additions in the list's order (no other rule, so out is their sum with the logit); with a
    temperature the same probabilities as the summed list gives."""
    V, P = 9001, 3
    rng = np.random.default_rng(B)
    toks = np.stack([rng.permutation(V)[:B] for _ in range(P)]).astype(np.int32)
    if kind == "one":
        toks[:, -1] = toks[:, 0]
    elif kind == "pairs":  # spread over the stretches, some three times, with ids outside the vocabulary between them
        toks[:, 2::3], toks[:, B // 2] = toks[:, :len(toks[0, 2::3])], -1
        toks[1, ::5] = 2 ** 31 - 1
    else:
        toks[:] = V - 1
    vals = (rng.standard_normal((P, B)) * 10.0 ** rng.integers(-3, 4, (P, B))).astype(np.float32)
    if kind == "zeros":
        vals[:] = -0.0
    call = Call(2, 3, V, FP, FP, history=0, bias=B, mask=False, tokens=False, temp=temp, extra=1, seed=3)
    temperature = call.rules.get("temperature")
    call.rules = dict(P=P, bias_tokens=toks, bias=vals)
    summed = np.full((P, V), -0.0, np.float32)
    for s in range(P):
        for t, v in zip(toks[s], vals[s]):
            if 0 <= t < V:
                summed[s, t] += v
    if temp:
        call.rules["temperature"] = temperature
        got, status = call.run()
        call.rules = dict(P=P, temperature=temperature)
        call.sh = call.sh._replace(max_bias=0)
        call.logits = call.logits + dev(summed[call.slots])[:, None]
        assert status == 0 and torch.equal(got.view(torch.int32), call.run()[0].view(torch.int32))
        return
    got, status = call.run()
    assert status == 0
    want = as_numpy(call.logits) + summed[call.slots][:, None]
    assert np.array_equal(as_numpy(got).view(np.int32), want.view(np.int32))


def test_a_token_twice_costs_little():
    """A list of 1024 biases with one token twice, and of one token throughout, beside one without (scans of the list in memory took
    47 times the whole call for either).  One token: a wave looks at 16 entries a lane.  All the same: 1024 additions in
    the list's order, each behind 8 dependent scalar and lane instructions of some 10 cycles, 1024 * 80 / 2.4 GHz = 34 us
    beside a call of 4 to 5 us."""
    C, V, B = 4, 32768, 1024
    call = Call(C, 1, V, BF, BF, history=0, bias=B, mask=False, tokens=False, tree=False, temp=False, extra=0, seed=4)
    out, slots, status = torch.empty(C, 1, V, dtype=BF, device="cuda"), dev(call.slots), torch.zeros(1, dtype=torch.int32, device="cuda")
    us = {}
    for kind in ("none", "one", "equal"):
        toks = np.stack([call.rng.permutation(V)[:B] for _ in range(C)]).astype(np.int32)
        if kind == "one":
            toks[:, -1] = toks[:, 0]
        if kind == "equal":
            toks[:] = 9
        toks, vals, times = dev(toks), dev(call.rules["bias"]), []
        for _ in range(7):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(50):
                gdn.adjust_logits(call.sh, call.logits, slots, bias_tokens=toks, bias=vals, out=out, status=status)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b) * 20)
        us[kind] = min(times)
    log(f"[logits] 1024 biases: {us} us")
    assert us["one"] < 3 * us["none"] and us["equal"] < 16 * us["none"]


@pytest.mark.parametrize("dtype,out", [(BF, FP), (BF, BF), (FP, FP), (HF, HF), (HF, FP)])
@pytest.mark.parametrize("temp", [None, 1.0, 0.0])
def test_every_value_beside_infinities_and_nan(dtype, out, temp):
    """Row by row: infinite and masked values exactly, finite ones within `expected`.

    The oracle's values are rounded to 32 bits where the type's lowest value is a row's: the call computes there (a penalty
    beside it is lost, a repetition of it overflows), and with bfloat16's or float32's the tolerance of `expected`, which is of
    the row's largest size, would be no test: all tokens that no rule touches have the same probability there."""
    call = Call(1, 8, 600, dtype, out, seed=7, temp=False, bias=3)
    s = call.slots[0]
    call.mask[:] = -1
    call.rules["repetition"][s], call.rules["bias_tokens"][s], call.rules["bias"][s] = 1.5, [50, 51, 52], [-np.inf, 1, 2]
    x = call.logits
    x[0, 0, 100] = x[0, 0, 200] = float("inf")
    x[0, 1, :] = -float("inf")
    x[0, 2, 77] = float("nan")
    x[0, 3, 33], x[0, 3, 34] = float("nan"), float("inf")
    call.mask[0, 3, 1], call.mask[0, 3, 9] = ~(3 << 1), 0x0F0F0F0F
    x[0, 4, 5] = -float("inf")
    call.mask[0, 4, 2:7] = 0x33333333
    x[0, 5, :] = float("nan")
    call.mask[0, 5] = 0
    x[0, 6, :] = torch.finfo(dtype).min
    call.mask[0, 7] = 0
    x[0, 7, :] = float("inf")
    if temp is not None:
        call.rules["temperature"] = np.full(call.sh.n_slots, temp, np.float32)
    got, status = call.run()
    res, bits = call.want()
    assert status == bits == 0
    g, word, at = as_numpy(got).astype(np.float64), np.arange(600) // 32, np.arange(600) % 32
    for i in range(8):
        z, size, T = res[0, i]
        masked = (call.mask[0, i].view(np.uint32)[word] >> at.astype(np.uint32)) & 1 == 0
        with np.errstate(over="ignore"):
            low = i == 6 and dtype is not HF
            z = z.astype(np.float32).astype(np.float64) if low else z
            want, tol = expected(z, size, T, call.sh)
            if low and T == 1.0:
                want = L.probabilities(z, T)
                assert np.count_nonzero(want) > 500 and len(np.unique(want)) == 2
                tol = want * (2.0 ** -19 + (2.0 ** -8 if out is BF else 0)) + 1e-35
            if T is None:  # beyond the type's range: an infinity of it
                want = np.where(np.abs(want) > float(torch.finfo(out).max) * (1 + 2.0 ** -12), np.sign(want) * np.inf, want)
        exact = masked | ~np.isfinite(want) | ~np.isfinite(z) | (T == 0) | ((T is not None) & (want == 0))
        assert np.array_equal(g[0, i][exact], want[exact], equal_nan=True), f"row {i}"
        fine = ~exact
        if fine.any():
            ratio = np.abs(g[0, i][fine] - want[fine]) / tol[fine]
            assert ratio.max() <= 1, f"row {i} is {ratio.max():.2f} tolerances off at {int(np.flatnonzero(fine)[np.argmax(ratio)])}"


def test_a_repetition_is_a_product_with_the_rounded_reciprocal():
    """As the header says, bit for bit: above zero fl(z fl(1 / r)), elsewhere fl(z r)."""
    V, P = 4500, 4
    call = Call(4, 1, V, FP, FP, history=V, bias=0, mask=False, tokens=False, tree=False, temp=False, extra=0, seed=5)
    r = np.array([1.1, 1.25, 3.0, 0.7], np.float32)
    call.rules = dict(P=P, history=np.tile(np.arange(V, dtype=np.int32), (P, 1)), history_len=np.full(P, V, np.int32),
                      prompt_len=np.full(P, V, np.int32), repetition=r)
    got, status = call.run()
    x, by = as_numpy(call.logits)[:, 0], r[call.slots][:, None]
    want = np.where(x > 0, x * (np.float32(1) / by), x * by)
    assert status == 0 and want.dtype == np.float32 and np.array_equal(as_numpy(got)[:, 0].view(np.int32), want.view(np.int32))
