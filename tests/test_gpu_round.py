"""Rotary cache write, draft acceptance and cache commit against the fp64 oracle, and a whole round of
an attention layer beside the recurrence's, as it would be used."""

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gpu_util import log
from oracle import gdn_oracle as O
from oracle import round_oracle as R
from round_util import HALF_STEP, SENTINEL, Paged, as_numpy, check_attention, dev, random_parents
from workloads import synth_case

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


# ---------------------------------------------------------------- rotary positions and the cache write
def _rope(pg, q, k, v, half, parents=None, nodes=None, slots=None, length=None, table=None, **kw):
    sh = pg.sh
    inv = 1e4 ** (-np.arange(half) / half)
    q_out = torch.full((sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim), SENTINEL, dtype=sh.dtype, device="cuda")
    s, t, n = (pg.slots if slots is None else slots, pg.table if table is None else table, pg.len if length is None else length)
    k64, v64 = as_numpy(pg.k).astype(np.float64), as_numpy(pg.v).astype(np.float64)
    before = k64.copy(), v64.copy()
    gpu = {a: None if b is None else dev(b) if isinstance(b, np.ndarray) else b for a, b in kw.items()}
    _, status = gdn.rope_kv_write(sh, q, k, v, dev(inv), pg.k, pg.v, dev(s), dev(t), dev(n),
                                  parents=None if parents is None else dev(parents),
                                  lane_nodes=None if nodes is None else dev(nodes), q_out=q_out, **gpu)
    torch.cuda.synchronize()
    pos = kw.get("positions")
    res, bits = R.rope_kv_write(as_numpy(q), as_numpy(k), as_numpy(v), inv, k64, v64, s, t, n, parents=parents,
                                lane_nodes=nodes, n_axes=1 if pos is None else pos.shape[2], **kw)
    assert int(status.item()) == bits
    # A turned value is a cos - b sin.  The angle's fraction of a turn is rounded to 32 bits (2^-25 of a turn),
    # sine and cosine to 2^-22, the two products and their difference to 2^-24 each: below 2^-20 (|a| + |b|).
    # The norm's sum of D squares and its root add (D + 4) 2^-24.  Then one rounding to the type.
    def near(got, want, mag):
        err = np.abs(got - want)
        tol = mag * (2.0 ** -19 + (sh.head_dim + 4) * 2.0 ** -24) + HALF_STEP[sh.dtype] * np.abs(want) * (1 + 2.0 ** -6) + 1e-30
        assert (err <= tol).all(), float(np.max(err / tol))

    got = as_numpy(q_out).astype(np.float64)
    for c in range(sh.n_seqs):
        for i in range(sh.n_nodes):
            if (c, i) in res:
                near(got[c, i], res[c, i], np.sqrt((res[c, i] ** 2).sum(-1, keepdims=True)))
            else:
                assert (got[c, i] == SENTINEL).all()
    for name, cache, want, old in (("k", pg.k, k64, before[0]), ("v", pg.v, v64, before[1])):
        g = as_numpy(cache).astype(np.float64)
        same = (want == old).all(-1)
        assert np.array_equal(g[same], old[same]), f"{name}: a row that is not the round's was written"
        near(g[~same], want[~same], np.sqrt((want[~same] ** 2).sum(-1, keepdims=True)))
    return res, bits


def _qkv(pg, xdtype):
    sh = pg.sh
    x = pg.normal(sh.n_seqs, sh.n_nodes, sh.n_q_heads + 2 * sh.n_kv_heads, sh.head_dim, dtype=xdtype)
    a, b = sh.n_q_heads, sh.n_q_heads + sh.n_kv_heads
    return x[:, :, :a], x[:, :, a:b], x[:, :, b:]


@pytest.mark.parametrize("xdtype,dtype", [(BF, BF), (HF, HF), (FP, FP), (FP, BF), (FP, HF)])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 16), (128, 128), (256, 64), (256, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_types_and_widths(xdtype, dtype, D, rot, interleaved):
    pg = Paged(2, 3, 6, 2, D, 16, dtype, [15, 40], seed=rot)
    _rope(pg, *_qkv(pg, xdtype), rot // 2, interleaved=interleaved)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_rope_axes_norms_trees_and_ragged_lanes(D):
    C, N = 3, 9
    pg = Paged(C, N, 5, 1, D, 7, BF, [0, 33, 12], seed=D)
    half = D // 4
    w = lambda: (1 + 0.2 * pg.rng.standard_normal(D)).astype(np.float32)  # noqa: E731
    parents, nodes = random_parents(pg.rng, C, N), np.array([N, 0, 4], np.int32)
    q, k, v = _qkv(pg, FP)
    _rope(pg, q, k, v, half, parents, nodes, q_norm=w(), k_norm=w(), eps=1e-5)
    _rope(pg, q, k, v, half, q_norm=None, k_norm=w(), eps=1e-5)
    _rope(pg, q, k, v, half, q_norm=w(), k_norm=None, eps=0.0)
    pos = pg.rng.integers(-5, 1 << 22, (C, N, 3)).astype(np.int32)
    axis = (np.arange(half) % 3).astype(np.int32)
    _rope(pg, q, k, v, half, positions=pos, pair_axis=axis)
    _rope(pg, q, k, v, half, positions=pos)  # every pair on axis 0


def test_rope_far_text_positions():
    """A text position of 10^6 and the page arithmetic at the end of a large table."""
    pg = Paged(1, 2, 2, 1, 64, 64, BF, [5], seed=3)
    sh = pg.sh._replace(max_pages=20000)
    table = np.full((sh.n_slots, 20000), -1, np.int32)
    length = pg.len.copy()
    length[pg.slots[0]] = 1_000_063  # the round's rows lie in entries 15625 and 15626
    table[pg.slots[0], 15625], table[pg.slots[0], 15626] = 0, 1
    pg.sh = sh
    _rope(pg, *_qkv(pg, FP), 32, table=table, length=length)


def test_rope_refuses_lanes_and_pages():
    C, N = 6, 3
    pg = Paged(C, N, 2, 1, 64, 4, BF, [6] * C, seed=4)
    slots, length, parents, nodes = pg.slots.copy(), pg.len.copy(), random_parents(pg.rng, C, N), np.full(C, N, np.int32)
    slots[1] = slots[0]  # both lanes are refused
    slots[2] = -3
    nodes[3] = -1
    parents[4, 1] = 1
    q, k, v = _qkv(pg, BF)
    res, bits = _rope(pg, q, k, v, 16, parents, nodes, slots=slots, length=length)
    assert bits == R.SLOT_DUP | R.SLOT_RANGE | R.NODES | R.PARENT and {c for c, _ in res} == {5}
    table = pg.table.copy()
    table[pg.slots[0], 2] = pg.sh.n_pages  # holds the last row of the round
    res, bits = _rope(pg, q, k, v, 16, table=table)
    assert bits == R.PAGE and len(res) == C * N
    _, bits = _rope(pg, q, k, v, 16, positions=np.zeros((C, N, 2), np.int32), pair_axis=np.full(16, 2, np.int32))
    assert bits == R.AXIS
    slots = np.full(C, -1, np.int32)
    res, bits = _rope(pg, q, k, v, 16, slots=slots)
    assert bits == 0 and not res


# ---------------------------------------------------------------- acceptance
def _probabilities(rng, shape, sharp=2.0):
    x = np.exp(sharp * rng.standard_normal(shape))
    return x / x.sum(-1, keepdims=True)


def _accept_inputs(C, N, V, dtype, tree, with_draft, with_root, seed):
    rng = np.random.default_rng(seed)
    p = _probabilities(rng, (C, N + 1, V))
    q = _probabilities(rng, (C, N, V)) * 0.3 + 0.7 * p[:, :N]
    parents = random_parents(rng, C, N) if tree else None
    target, root = dev(p[:, 1:].astype(np.float32), dtype), dev(p[:, 0].astype(np.float32), dtype) if with_root else None
    draft = dev(q.astype(np.float32), dtype) if with_draft else None
    tokens = np.empty((C, N), np.int32)
    for c in range(C):
        for i in range(N):
            par = i - 1 if parents is None else parents[c, i]
            row = q[c, i] if with_draft else p[c, par + 1]
            tokens[c, i] = rng.choice(V, p=row / row.sum()) if rng.random() < 0.8 else rng.integers(V)
    u, u_next = rng.random((C, N), dtype=np.float32), rng.random(C, dtype=np.float32)
    return target, root, draft, tokens, parents, u, u_next


def _accept(target, root, draft, tokens, parents, u, u_next, nodes=None, slots=None, greedy=False):
    C, N, V = target.shape
    sh = gdn.AcceptShape(C, N, V, target.dtype)
    ws = torch.full((gdn.draft_accept_workspace_size(sh) // 4,), float("nan"), device="cuda")
    outs = [torch.full((C,), -77, dtype=torch.int32, device="cuda") for _ in range(3)]
    g = lambda a: None if a is None else dev(a)  # noqa: E731
    *_, status = gdn.draft_accept(sh, target, dev(tokens), root_target=root, draft=draft, parents=g(parents), lane_nodes=g(nodes),
                                  slot_ids=g(slots), u_accept=None if greedy else dev(u), u_next=None if greedy else dev(u_next),
                                  accept_node=outs[0], n_accept=outs[1], next_token=outs[2], workspace=ws)
    torch.cuda.synchronize()
    f = lambda t: None if t is None else as_numpy(t)  # noqa: E731
    res, bits = R.draft_accept(f(target), tokens, f(root), f(draft), parents, nodes, slots, None if greedy else u,
                               None if greedy else u_next)
    got = np.stack([o.cpu().numpy() for o in outs], 1)
    assert int(status.item()) == bits
    for c in range(C):
        assert tuple(got[c]) == res.get(c, (-77, -77, -77)), f"lane {c}: {got[c]} against {res.get(c)}"
    return got, bits


@pytest.mark.parametrize("dtype", [FP, BF, HF])
@pytest.mark.parametrize("V", [1, 2, 33, 4095, 4096, 4097, 50001])
@pytest.mark.parametrize("mode,tree", [("draft", False), ("candidates", False), ("candidates", True), ("greedy", False),
                                       ("greedy", True)])
def test_accept_against_the_oracle(dtype, V, mode, tree):
    for seed, (C, N, root) in enumerate([(5, 7, True), (3, 32, False), (4, 1, False), (4, 1, True)]):
        args = _accept_inputs(C, N, V, dtype, tree, mode == "draft", root, 100 * V + seed)
        nodes = np.random.default_rng(seed).integers(0, N + 1, C).astype(np.int32) if seed == 0 else None
        got, _ = _accept(*args, nodes=nodes, greedy=mode == "greedy")
        log(f"[accept] {dtype} V={V} {mode} tree={tree} C={C} N={N}: accepted {got[:, 1].tolist()}")


def test_accept_limits():
    """Everything accepted, everything refused, the last token, duplicate candidates, rows without weight."""
    C, N, V = 4, 3, 5000
    target, root, _, tokens, _, u, u_next = _accept_inputs(C, N, V, FP, False, False, True, 1)
    got, _ = _accept(target, root, None, tokens, None, np.zeros_like(u), u_next)
    assert (got[:, 1] == N).all()
    got, _ = _accept(target, root, None, tokens, None, np.full_like(u, 1 - 2.0 ** -24), np.full_like(u_next, 1 - 2.0 ** -24))
    assert (got[:, 0] == -1).all() and (got[:, 2] > V - 200).all()
    got, _ = _accept(target, root, None, tokens, None, u, np.zeros_like(u_next))
    q = target.clone()  # the draft is the target: never refused
    chain = torch.cat((root[:, None], target[:, :-1]), 1).contiguous()
    got, _ = _accept(target, root, chain, tokens, None, np.full_like(u, 1 - 2.0 ** -24), u_next)
    assert (got[:, 1] == N).all()
    parents = np.array([[-1, -1, -1]] * C, np.int32)
    same = np.tile(tokens[:, :1], (1, 3))
    _accept(target, root, None, same, parents, np.full_like(u, 0.999), u_next)
    none = torch.zeros_like(target)
    got, _ = _accept(none, torch.zeros_like(root), None, tokens, None, u, u_next)
    assert (got[:, 2] == -1).all()
    one = torch.zeros_like(root)
    one[:, 4096] = 0.5  # a single weight, which refusing it removes: drawn all the same
    got, _ = _accept(none, one, None, np.full((C, N), 4096, np.int32), None, np.full_like(u, 0.75), u_next)
    assert (got[:, 0] == -1).all() and (got[:, 2] == 4096).all()
    odd = root.clone()
    odd[:, ::3] = float("nan")
    odd[:, 1::3] = -1.0
    _accept(target, odd, None, tokens, None, u, u_next)
    _accept(odd[:, None].expand(C, N, V).contiguous(), None, None, tokens, None, u, u_next, greedy=True)
    flat = torch.full_like(target, float("nan"))
    got, _ = _accept(flat, None, None, tokens, None, u, u_next, greedy=True)
    ties = torch.zeros_like(target)
    got, _ = _accept(ties, None, None, np.zeros_like(tokens), None, u, u_next, greedy=True)
    assert (got[:, 0] == N - 1).all() and (got[:, 2] == 0).all()
    del q


def test_accept_refuses_lanes():
    C, N, V = 6, 4, 300
    target, root, _, tokens, parents, u, u_next = _accept_inputs(C, N, V, FP, True, False, True, 2)
    slots, nodes = np.arange(C).astype(np.int32), np.full(C, N, np.int32)
    slots[0] = -1
    nodes[1] = N + 1
    parents[2, 3] = 3
    tokens[3, 1] = V
    nodes[4], tokens[4, 3] = 3, -9  # an absent node's token is not looked at
    for greedy in (False, True):
        got, bits = _accept(target, root, None, tokens, parents, u, u_next, nodes, slots, greedy)
        assert bits == R.NODES | R.PARENT | R.TOKEN
        assert (got[:4] == -77).all() and (got[4:] != -77).all()


def test_accept_leaves_the_targets_distribution():
    """A refused or accepted first token has the target's distribution: over a grid of random numbers the share of
    each token is its probability, within the grid's step for each of the V + 1 borders a cell may straddle."""
    V, n = 4, 64
    p, q = np.array([0.5, 0.2, 0.2, 0.1], np.float32), np.array([0.1, 0.6, 0.1, 0.2], np.float32)
    share = np.zeros(V)
    grid = ((np.arange(n) + 0.5) / n).astype(np.float32)
    ua, un = (g.ravel() for g in np.meshgrid(grid, grid, indexing="ij"))
    for t in range(V):
        for lo in range(0, n * n, 1024):
            u, w = ua[lo:lo + 1024, None], un[lo:lo + 1024]
            C = len(w)
            target, root = dev(np.tile(p, (C, 1, 1))), dev(np.tile(p, (C, 1)))
            got, _ = _accept(target, root, dev(np.tile(q, (C, 1, 1))), np.full((C, 1), t, np.int32), None, u, w)
            first = np.where(got[:, 0] == 0, t, got[:, 2])
            share += q[t] * np.bincount(first, minlength=V) / (n * n)
    assert (np.abs(share - p) <= (V + 1) / n).all(), share


# ---------------------------------------------------------------- commit
def _commit(pg, accept, parents, nodes=None, status_in=0, slots=None, table=None, length=None, as_list=False):
    s, t, n = (pg.slots if slots is None else slots, pg.table if table is None else table, pg.len if length is None else length)
    status = torch.full((1,), status_in, dtype=torch.int32, device="cuda")
    k, v = as_numpy(pg.k), as_numpy(pg.v)
    new_len, bits = R.kv_commit(list(k), list(v), s, t, n, accept, parents, nodes, status_in, N=pg.sh.n_nodes)
    kk, vv = (list(pg.k), list(pg.v)) if as_list else (pg.k, pg.v)
    got = gdn.kv_commit_layers(pg.sh, kk, vv, dev(s), dev(t), dev(n), dev(accept), status,
                               parents=None if parents is None else dev(parents), lane_nodes=None if nodes is None else dev(nodes))
    torch.cuda.synchronize()
    assert int(status.item()) == bits
    assert np.array_equal(got.cpu().numpy(), new_len)
    assert np.array_equal(as_numpy(pg.k), k) and np.array_equal(as_numpy(pg.v), v)
    return bits


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,Hkv,page,N", [(64, 1, 1, 32), (128, 3, 5, 16), (256, 8, 64, 32), (128, 2, 16, 1)])
def test_commit_moves_rows(dtype, D, Hkv, page, N):
    C = 5
    pg = Paged(C, N, Hkv, Hkv, D, page, dtype, [0, 1, 17, 64, 100], seed=D + N, layers=3)
    parents = random_parents(pg.rng, C, N)
    accept = pg.rng.integers(-1, N, C).astype(np.int32)
    accept[0], accept[1] = N - 1, -1
    assert _commit(pg, accept, parents, as_list=page == 5) == 0
    chain = np.tile(np.arange(-1, N - 1, dtype=np.int32), (C, 1))
    assert _commit(pg, accept, chain) == 0
    nodes = np.minimum(accept + 1 + pg.rng.integers(0, 3, C), N).astype(np.int32)
    assert _commit(pg, accept, random_parents(pg.rng, C, N), nodes) == 0


def test_commit_of_a_chain_only_advances_lengths():
    pg = Paged(3, 500, 2, 2, 64, 16, BF, [0, 5, 40], seed=5, layers=2)
    assert _commit(pg, np.array([499, -1, 0], np.int32), None) == 0


def test_commit_is_a_transaction():
    C, N = 4, 6
    pg = Paged(C, N, 2, 2, 64, 8, BF, [9, 20, 3, 30], seed=6, layers=2)
    parents, accept = random_parents(pg.rng, C, N), np.array([5, 3, 4, 2], np.int32)
    ok = dict(parents=parents, accept=accept)

    def bad(bit, **kw):
        assert _commit(pg, **{**ok, **kw}) == bit

    bad(1024, status_in=1024)
    slots = pg.slots.copy()
    slots[2] = pg.sh.n_slots
    bad(R.SLOT_RANGE, slots=slots)
    slots[2] = slots[1]
    bad(R.SLOT_DUP, slots=slots)
    p = parents.copy()
    p[3, 4] = 5
    bad(R.PARENT, parents=p)
    bad(R.ACCEPT, accept=np.array([5, 3, 6, 2], np.int32))
    bad(R.ACCEPT, accept=np.array([5, 3, -2, 2], np.int32))
    bad(R.ACCEPT, nodes=np.array([6, 3, 6, 6], np.int32))
    bad(R.NODES, nodes=np.array([6, 6, 7, 6], np.int32))
    length = pg.len.copy()
    length[pg.slots[0]] = pg.sh.max_pages * 8
    bad(R.LENGTH, length=length)
    table = pg.table.copy()
    table[pg.slots[1], 20 // 8] = -1
    bad(R.PAGE, table=table)
    slots = pg.slots.copy()
    slots[1] = -1  # padding: nothing of it is looked at
    assert _commit(pg, accept, parents, slots=slots, table=table) == 0


def test_write_and_commit_past_32_bits():
    """Pools of more than 2^32 bytes: rows are written and moved where they lie, as in a small pool."""
    page, D, Hkv, N, L = 128, 256, 4, 6, 250
    per = Hkv * page * D * 2
    n_pages = (1 << 32) // per + 40
    small = Paged(1, N, 8, Hkv, D, page, BF, [L], seed=21, extra_slots=0, spare_pages=0)
    sh = small.sh._replace(n_pages=n_pages)
    ids = np.array([[3, n_pages - 1]], np.int32)
    k, v = (torch.zeros(sh.cache_shape, dtype=BF, device="cuda") for _ in range(2))
    for big, of in ((k, small.k), (v, small.v)):
        for j in range(2):
            big[int(ids[0, j])] = of[int(small.table[0, j])]
    q_, k_, v_ = _qkv(small, BF)
    inv, (slots, table, length) = dev(1e4 ** (-np.arange(64) / 64)), small.places()
    parents = dev(np.array([[-1, 0, 0, 1, 2, 3]], np.int32))
    accept = dev(np.array([5], np.int32))  # nodes 0, 1, 3, 5: rows L + 3 and L + 5 move to L + 2 and L + 3
    for sh_, kk, vv, tab in ((small.sh, small.k, small.v, table), (sh, k, v, dev(ids))):
        _, status = gdn.rope_kv_write(sh_, q_, k_, v_, inv, kk, vv, slots, tab, length, parents=parents)
        gdn.kv_commit_layers(sh_, [kk], [vv], slots, tab, length, accept, status, parents=parents)
        assert int(status.item()) == 0
    for big, of in ((k, small.k), (v, small.v)):
        for j in range(2):
            assert torch.equal(big[int(ids[0, j])], of[int(small.table[0, j])])


def test_most_lanes_of_the_write_and_the_commit():
    C, N = 1024, 7
    pg = Paged(C, N, 2, 1, 64, 16, BF, [c % 40 for c in range(C)], seed=22)
    parents, nodes = random_parents(pg.rng, C, N), pg.rng.integers(1, N + 1, C).astype(np.int32)
    slots = pg.slots.copy()
    slots[::9] = -1
    res, bits = _rope(pg, *_qkv(pg, BF), 32, parents, nodes, slots=slots)
    assert bits == 0 and len(res) == int(nodes[slots >= 0].sum())
    pg.k, pg.v = pg.k[None].contiguous(), pg.v[None].contiguous()
    accept = np.minimum(pg.rng.integers(-1, N, C), nodes - 1).astype(np.int32)
    assert _commit(pg, accept, parents, nodes, slots=slots) == 0
    again = slots.copy()
    again[1023] = again[1]  # the last lane and one of the first
    assert _commit(pg, accept, parents, nodes, slots=again) == R.SLOT_DUP


# ---------------------------------------------------------------- a round, as it is used
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("sharp", [1.0, 4.0])
def test_a_round_of_both_layer_kinds(graph, sharp):
    """Three rounds without host synchronisation: rotation and cache write, attention over the draft tree, the
    recurrence's verify on the same tree, acceptance on the device, and both commits by its accept_node.  Flat
    target distributions refuse every candidate, sharp ones accept paths of several nodes."""
    C, N, V, Hq, Hkv, D, page = 3, 12, 997, 4, 2, 64, 16
    rounds = 3
    pg = Paged(C, rounds * N, Hq, Hkv, D, page, FP, [21, 0, 50], seed=7, layers=1)
    sh = pg.sh._replace(n_nodes=N)
    case = synth_case(C, N, pg.sh.n_slots, 2, 4, 64, 64, seed=8, tree=True)
    gsh = gdn.Shape(C, N, pg.sh.n_slots, 2, 4, 64, 64)
    rng = pg.rng
    inv = 1e4 ** (-np.arange(32) / 32)
    feed = []
    for r in range(rounds):
        parents = random_parents(rng, C, N)
        p = _probabilities(rng, (C, N + 1, V), sharp)
        tokens = np.empty((C, N), np.int32)
        for c in range(C):
            for i in range(N):
                tokens[c, i] = int(np.argmax(p[c, parents[c, i] + 1])) if rng.random() < 0.7 else rng.integers(V)
        feed.append(dict(parents=parents, target=p[:, 1:].astype(np.float32), root=p[:, 0].astype(np.float32), tokens=tokens,
                         x=rng.standard_normal((C, N, Hq + 2 * Hkv, D)).astype(np.float32),
                         gx=rng.standard_normal(case["x"].shape).astype(np.float32),
                         u=(0.3 * rng.random((C, N))).astype(np.float32), un=rng.random(C, dtype=np.float32)))
    # device side: fixed buffers, refilled before every round
    buf = {k: dev(v) for k, v in feed[0].items()}
    state, hist, ba = dev(case["state"]), dev(case["conv_hist"]), dev(case["ba"])
    conv_w, dt_bias, A = dev(case["conv_w"]), dev(case["dt_bias"]), dev(case["A"])
    slots, table, length = pg.places()
    k0, v0, s0, h0, l0 = pg.k.clone(), pg.v.clone(), state.clone(), hist.clone(), length.clone()
    new_len = torch.zeros_like(length)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, att = (torch.zeros(C, N, Hq, D, device="cuda") for _ in range(2))
    ws = torch.empty(max(1, gdn.paged_attention_workspace_size(sh) // 4), device="cuda")
    ash = gdn.AcceptShape(C, N, V, FP)
    aws = torch.empty(gdn.draft_accept_workspace_size(ash) // 4, device="cuda")
    acc = [torch.zeros(C, dtype=torch.int32, device="cuda") for _ in range(3)]
    inv_d = dev(inv)
    outs = dict(out=torch.zeros(C, N, 4, 64, device="cuda"), log=torch.zeros(C, N, 4, gsh.log_row, device="cuda"),
                win=torch.zeros(C, N, gsh.channels, 3, device="cuda"))

    def one_round():
        x = buf["x"]
        gdn.rope_kv_write(sh, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], inv_d, pg.k[0], pg.v[0], slots, table,
                          length, parents=buf["parents"], q_out=q_out, status=status)
        gdn.paged_attention(sh, q_out, pg.k[0], pg.v[0], slots, table, length, parents=buf["parents"], out=att, workspace=ws,
                            status=status)
        gdn.conv_tree_verify(gsh, buf["gx"], conv_w, hist, ba[..., :4], ba[..., 4:], dt_bias, A, state, slots, buf["parents"],
                             out=outs["out"], replay_log=outs["log"], commit_win=outs["win"], status=status)
        gdn.draft_accept(ash, buf["target"], buf["tokens"], root_target=buf["root"], parents=buf["parents"], slot_ids=slots,
                         u_accept=buf["u"], u_next=buf["un"], accept_node=acc[0], n_accept=acc[1], next_token=acc[2],
                         workspace=aws, status=status)
        gdn.replay_commit(gsh, outs["log"], outs["win"], slots, buf["parents"], acc[0], state, hist, status)
        gdn.kv_commit_layers(sh, pg.k, pg.v, slots, table, length, acc[0], status, parents=buf["parents"], new_len=new_len)
        length.copy_(new_len)

    def reset():
        for a, b in ((pg.k, k0), (pg.v, v0), (state, s0), (hist, h0), (length, l0)):
            a.copy_(b)

    replay = one_round
    if graph:
        one_round()  # warms up
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one_round()
        reset()
        replay = g.replay
    saved = []
    for r in range(rounds):
        for key, v in feed[r].items():
            buf[key].copy_(dev(v))
        replay()
        saved.append((att.clone(), acc[0].clone(), acc[2].clone(), length.clone()))
    torch.cuda.synchronize()
    assert int(status.item()) == 0

    # the oracle's rounds on the same inputs
    k64, v64 = as_numpy(k0[0]).astype(np.float64), as_numpy(v0[0]).astype(np.float64)
    pool, h64, lens = case["state"].astype(np.float64), case["conv_hist"].astype(np.float64), as_numpy(l0)
    moved = 0
    for r in range(rounds):
        f = feed[r]
        x = f["x"]
        qs, _ = R.rope_kv_write(x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], inv, k64, v64, pg.slots, pg.table,
                                lens, parents=f["parents"])
        q64 = np.stack([np.stack([qs[c, i] for i in range(N)]) for c in range(C)])
        res, _ = R.paged_attention(q64, k64, v64, pg.slots, pg.table, lens, parents=f["parents"])
        for (c, i), (out, mag, big, rows) in res.items():
            # rotated q and k are off by 2^-19 of their norm, scores so by 2^-18 big, weights by twice that
            tol = mag * (2.0 ** -16 * (1 + big) + (rows + 80) * 2.0 ** -22)
            err = np.abs(as_numpy(saved[r][0])[c, i] - out)
            assert (err <= tol).all(), (r, c, i, float(np.max(err / tol)))
        got, _ = R.draft_accept(f["target"], f["tokens"], f["root"], None, f["parents"], u_accept=f["u"], u_next=f["un"])
        accept = np.array([got[c][0] for c in range(C)], np.int32)
        assert np.array_equal(as_numpy(saved[r][1]), accept)
        assert np.array_equal(as_numpy(saved[r][2]), [got[c][2] for c in range(C)])
        ref = O.verify_round(f["gx"], case["ba"], case["conv_w"], h64, pool, case["dt_bias"], case["A"], pg.slots, f["parents"], 2, None)
        assert O.replay_commit(ref["replay_log"], ref["commit_win"], pg.slots, f["parents"], accept, pool, h64, 0, None) == 0
        lens, _ = R.kv_commit([k64], [v64], pg.slots, pg.table, lens, accept, f["parents"])
        assert np.array_equal(as_numpy(saved[r][3]), lens)
        moved += sum(len(R.path_of(f["parents"][c], a)) for c, a in enumerate(accept) if a >= 0)
    assert moved > C if sharp > 1 else moved == 0  # the rounds do accept
    e = np.max(np.abs(as_numpy(state) - pool) / np.maximum(1.0, np.abs(pool)))
    assert e <= rounds * 2e-4, e  # the recurrence's own tolerance, per round
    for c in range(C):  # committed rows of the cache: rotated keys and copied values
        for t in range(int(lens[pg.slots[c]])):
            pid, at = int(pg.table[pg.slots[c], t // page]), t % page
            kk = k64[pid, :, at]
            assert (np.abs(as_numpy(pg.k[0, pid, :, at]) - kk) <= 2.0 ** -18 * np.sqrt((kk ** 2).sum(-1, keepdims=True))).all()
            assert np.array_equal(as_numpy(pg.v[0, pid, :, at]), v64[pid, :, at].astype(np.float32))
