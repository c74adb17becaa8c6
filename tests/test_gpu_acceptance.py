"""The acceptance on the device: the order of rows that hold NaN and infinities."""

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from round_util import dev

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("V", [3, 4096, 9001])
def test_greedy_ranks_nan_below_minus_infinity(dtype, V):
    """The largest value of a row: a NaN only where all are, minus infinity only where nothing else is, the lowest index."""
    nan, inf = float("nan"), float("inf")
    rows = np.full((7, V), -inf, np.float32)
    rows[0, 0] = nan
    rows[1, :-1] = nan
    rows[2] = nan
    rows[3, 1] = nan
    rows[4, :2], rows[4, -1] = (nan, -5.0), inf
    rows[5, :-1], rows[5, -1] = nan, -1.0
    want = np.array([1, V - 1, 0, 0, V - 1, V - 1, 0])
    tokens = np.full((7, 1), V - 1, np.int32)
    node, count, token, status = gdn.draft_accept(gdn.AcceptShape(7, 1, V, dtype), dev(rows[:, None], dtype), dev(tokens),
                                                  root_target=dev(rows, dtype))
    assert int(status.item()) == 0
    assert np.array_equal(token.cpu().numpy(), want)
    assert np.array_equal(node.cpu().numpy(), np.where(want == V - 1, 0, -1))
    assert np.array_equal(count.cpu().numpy(), (want == V - 1).astype(np.int32))
