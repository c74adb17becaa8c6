"""Pins of the acceptance oracle: the order of rows that hold NaN and infinities."""

import numpy as np

from oracle import round_oracle as R


def test_greedy_ranks_nan_below_minus_infinity():
    nan, inf = float("nan"), float("inf")
    rows = np.array([[nan, -inf, -inf], [nan, nan, -inf], [nan, nan, nan], [-inf, nan, -inf], [nan, -5.0, inf]], np.float32)
    res, _ = R.draft_accept(rows[:, None], np.full((5, 1), 2), root=rows)
    # the token 2 is accepted where it is the largest; the next token comes from an equal row
    assert [res[c] for c in range(5)] == [(-1, 0, 1), (0, 1, 2), (-1, 0, 0), (-1, 0, 0), (0, 1, 2)]
