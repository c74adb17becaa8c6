"""The acceptance rule leaves the target's distribution: the fp64 oracle integrated exactly over its random numbers, for
candidates and for drawn drafts; and the integration notices each term of the rule that is left out."""

import inspect
import types

import numpy as np
import pytest

import acceptance_util as A
from oracle import round_oracle as R


def _results(case, oracle=R):
    out = []
    for b in case.blocks(case.C):
        res, bits = oracle.draft_accept(b["target"], b["tokens"], b["root"], b["draft"], b["parents"], u_accept=b["u"], u_next=b["u_next"])
        assert bits == 0
        out += [res[c] for c in range(case.C)]
    return np.array(out)


def _deviations(oracle=R):
    """Largest deviation of the siblings' cases, of the drawn token, and of the drawn chain."""
    sib = max(np.abs(A.share_of_siblings(cand, case, _results(case, oracle)) - A.P).max() for cand, case in A.siblings())
    one = np.abs(sum(A.share_of_drawn(t, case, _results(case, oracle)) for t, case in A.drawn()) - A.P).max()
    first, second = (sum(s) for s in zip(*(A.shares_of_chain(p, case, _results(case, oracle)) for p, case in A.drawn_chain())))
    # an accepted first token leaves the second one p2, whatever it is
    return sib, one, max(np.abs(first - A.P).max(), np.abs(second / second.sum() - A.P2).max())


def test_the_first_tokens_are_the_targets():
    # (sums of at most 240 equal shares a case, off by 2^-53 each)
    assert max(_deviations()) < 1e-10


def _planted(old, new):
    """The oracle with one line of its acceptance changed."""
    text = inspect.getsource(R)
    assert text.count(old) == 1
    m = types.ModuleType("planted")
    exec(compile(text.replace(old, new), "planted", "exec"), m.__dict__)
    return m


@pytest.mark.parametrize("old,new,which", [
    ("left -= p[t] if p is not None else 0.0", "pass", 0),                           # siblings tested against p alone
    ("elif t in refused:", "elif False:", 0),                                        # a candidate twice
    ("w[refused] = 0.0", "pass", 0),                                                 # refused candidates drawn again
    ("w = np.maximum(p - np.where(qd > 0, qd, 0.0), 0.0)", "pass", 1),               # a refusal followed by a draw from p
    ("* qq * left < p[t]", "* left < p[t]", 1),                                      # the drafter's probability left out
    ("qd = draft[c, kids[0]]", "qd = draft[c, 0]", 2),                               # another node's draft row
])
def test_a_term_left_out_is_noticed(old, new, which):
    assert _deviations(_planted(old, new))[which] > 1e-3


def test_greedy_ranks_nan_below_minus_infinity():
    nan, inf = float("nan"), float("inf")
    rows = np.array([[nan, -inf, -inf], [nan, nan, -inf], [nan, nan, nan], [-inf, nan, -inf], [nan, -5.0, inf]], np.float32)
    res, _ = R.draft_accept(rows[:, None], np.full((5, 1), 2), root=rows)
    # the token 2 is accepted where it is the largest; the next token comes from an equal row
    assert [res[c] for c in range(5)] == [(-1, 0, 1), (0, 1, 2), (-1, 0, 0), (-1, 0, 0), (0, 1, 2)]
