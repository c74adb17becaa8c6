"""The acceptance on the device: its distribution integrated exactly over the random numbers, and the order of rows that
hold NaN and infinities."""

import numpy as np
import pytest
import torch

import acceptance_util as A
import gated_deltanet_speculative_amd as gdn
from gpu_util import log
from round_util import dev

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _results(case, dtype):
    """(accept_node, n_accept, next_token) of every lane; every probability is exact in each type."""
    out = []
    g = lambda a, t=None: None if a is None else dev(a, t)  # noqa: E731
    for b in case.blocks(1024):
        C, N, V = b["target"].shape
        *got, status = gdn.draft_accept(gdn.AcceptShape(C, N, V, dtype), g(b["target"], dtype), g(b["tokens"]),
                                        root_target=g(b["root"], dtype), draft=g(b["draft"], dtype), parents=g(b["parents"]),
                                        u_accept=g(b["u"]), u_next=g(b["u_next"]))
        assert int(status.item()) == 0
        out.append(np.stack([t.cpu().numpy() for t in got], 1))
    return np.concatenate(out)


@pytest.mark.parametrize("dtype", [FP, BF, HF])
def test_candidates_leave_the_targets_distribution(dtype):
    for cand, case in A.siblings():
        share = A.share_of_siblings(cand, case, _results(case, dtype))
        log(f"[accept] candidates {cand}, {case.C} lanes: {share.tolist()}")
        assert np.abs(share - A.P).max() < 1e-10, cand


@pytest.mark.parametrize("dtype", [FP, BF, HF])
def test_drawn_drafts_leave_the_targets_distribution(dtype):
    share = sum(A.share_of_drawn(t, case, _results(case, dtype)) for t, case in A.drawn())
    assert np.abs(share - A.P).max() < 1e-10
    first, second = (sum(s) for s in zip(*(A.shares_of_chain(p, case, _results(case, dtype)) for p, case in A.drawn_chain())))
    log(f"[accept] drawn {share.tolist()}, chain {first.tolist()} {(second / second.sum()).tolist()}")
    assert np.abs(first - A.P).max() < 1e-10 and np.abs(second / second.sum() - A.P2).max() < 1e-10


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
