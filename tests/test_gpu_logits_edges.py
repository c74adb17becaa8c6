"""Edges of the logits' rules on the GPU against the fp64 oracle: temperatures that are no normal numbers."""

import numpy as np
import pytest

from gpu_util import log
from oracle import logits_oracle as L
from round_util import as_numpy, dev
from test_gpu_logits import FP, Call

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
