"""Cases in which the acceptance can be integrated exactly over its random numbers.

Every probability is a small fraction, so every threshold of a test or draw (p(x) / q(x), p(x') / (1 - p(x)), the running
sums of a residual) is a multiple of 1 / n for the number n of cells that the case names: over the cells' midpoints the
share of each outcome is its probability, without an error of the grid.  Each threshold lies half a cell from the nearest
midpoint, so no rounding of a number decides a test.
"""

from __future__ import annotations

import itertools

import numpy as np

P = np.array([8, 4, 2, 2]) / 16.0


class Case:
    """Lanes over all midpoints; `weight[c]` is the measure of lane c, `first` maps a result to the first token."""

    def __init__(self, root, target, tokens, u_cells, next_cells, draft=None, parents=None, weight=1.0):
        mids = [(np.arange(n) + 0.5) / n for n in (*u_cells, next_cells)]
        u = np.array(list(itertools.product(*mids)))
        self.C, self.N = len(u), len(tokens)
        lanes = lambda a: None if a is None else np.ascontiguousarray(np.broadcast_to(a, (self.C, *np.shape(a))))  # noqa: E731
        self.root, self.target, self.draft = lanes(np.float32(root)), lanes(np.float32(target)), lanes(None if draft is None else np.float32(draft))
        self.tokens, self.parents = lanes(np.int32(tokens)), lanes(None if parents is None else np.int32(parents))
        self.u, self.u_next, self.weight = u[:, :-1].astype(np.float32), u[:, -1].astype(np.float32), weight / self.C

    def blocks(self, lanes):
        """The lanes in blocks, as keyword arguments of the acceptance."""
        for lo in range(0, self.C, lanes):
            s = slice(lo, lo + lanes)
            cut = lambda a: None if a is None else a[s]  # noqa: E731
            yield dict(target=self.target[s], root=self.root[s], draft=cut(self.draft), tokens=self.tokens[s],
                       parents=cut(self.parents), u=self.u[s], u_next=self.u_next[s])


def siblings():
    """Candidates of the prefix in each order: the first token's distribution is P, whichever they are."""
    target = np.tile(P, (3, 1))
    for cand, cells, nxt in (
            ([0, 1], (4, 4), 4),        # tests 1/2, 1/2; draw of {2, 3} 1/2
            ([1, 0], (4, 6), 4),        # tests 1/4, 2/3; draw of {2, 3} 1/2
            ([1, 2], (4, 6), 10),       # tests 1/4, 1/6; draw of {0, 3} 4/5
            ([2, 2], (8, 14), 14),      # test 1/8, the second refused (1/7 if it were not); draw of {0, 1, 3} 4/7, 6/7
            ([0, 1, 2], (4, 4, 4), 2),  # tests 1/2, 1/2, 1/2; draw of {3}
            ([0, 2, 1], (4, 4, 6), 2),  # tests 1/2, 1/4, 2/3; draw of {3}
            ([1, 0, 3], (4, 6, 4), 2)):  # tests 1/4, 2/3, 1/2; draw of {2}
        n = len(cand)
        yield cand, Case(P, target[:n], cand, cells, nxt, parents=[-1] * n)


def drawn(q=np.array([4, 8, 1, 3]) / 16.0):
    """A token drawn from q, for each of its values: together the first token's distribution is P.  Thresholds p / q: 1/2
    and 2/3; max(p - q, 0) is 4/16 and 1/16, whose draw has the threshold 4/5."""
    for t in range(4):
        yield t, Case(P, [P], [t], (6,), 10, draft=[q], weight=q[t])


def drawn_chain():
    """Two tokens drawn from q and q2: pairs of first and second token (the second after an accepted first one, thresholds
    p2 / q2 1/2 and 3/4; max(p2 - q2, 0) is one token)."""
    q, q2, p2 = np.array([4, 8, 1, 3]) / 16.0, np.array([2, 2, 8, 4]) / 16.0, np.array([1, 6, 6, 3]) / 16.0
    for t, t2 in itertools.product(range(4), range(4)):
        yield (t, t2), Case(P, [p2, P], [t, t2], (6, 4), 10, draft=[q, q2], weight=q[t] * q2[t2])


P2 = np.array([1, 6, 6, 3]) / 16.0


def share_of_siblings(cand, case, results):
    """Share of each first token; results: (accept_node, n_accept, next_token) of every lane."""
    node, token = results[:, 0], results[:, 2]
    first = np.where(node >= 0, np.asarray(cand)[node], token)
    return np.bincount(first, minlength=4) * case.weight


def share_of_drawn(t, case, results):
    return np.bincount(np.where(results[:, 0] == 0, t, results[:, 2]), minlength=4) * case.weight


def shares_of_chain(pair, case, results):
    """Shares of the first token, and of the second token where the first was accepted."""
    first = np.where(results[:, 0] >= 0, pair[0], results[:, 2])
    second = np.where(results[:, 0] == 1, pair[1], results[:, 2])
    went = results[:, 0] >= 0
    return np.bincount(first, minlength=4) * case.weight, np.bincount(second[went], minlength=4) * case.weight
