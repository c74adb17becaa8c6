"""Attention over the paged cache against the fp64 oracle: types, head layouts, page sizes, lengths
from one token, ragged and padded lanes, draft trees, gates, and whatever may lie in rows that a
node does not attend to."""

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gpu_util import log
from oracle import round_oracle as R
from round_util import SENTINEL, Paged, as_numpy, check_attention, dev, random_parents

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _run(pg, q, parents=None, lane_nodes=None, gate=None, gate_mode=1, scale=None, slots=None, table=None, length=None):
    sh = pg.sh
    out = torch.full((sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim), SENTINEL, dtype=sh.dtype, device="cuda")
    ws = torch.full((max(gdn.paged_attention_workspace_size(sh) // 4, 1),), float("nan"), device="cuda")
    s, t, n = (pg.slots if slots is None else slots, pg.table if table is None else table, pg.len if length is None else length)
    _, status = gdn.paged_attention(sh, q, pg.k, pg.v, dev(s), dev(t), dev(n),
                                    parents=None if parents is None else dev(parents),
                                    lane_nodes=None if lane_nodes is None else dev(lane_nodes), gate=gate,
                                    gate_mode=gate_mode, scale=scale, out=out, workspace=ws)
    torch.cuda.synchronize()
    res, bits = R.paged_attention(as_numpy(q), as_numpy(pg.k), as_numpy(pg.v), s, t, n, parents, lane_nodes, scale,
                                  None if gate is None else as_numpy(gate), gate_mode)
    return out, res, int(status.item()), bits


def _case(C, N, Hq, Hkv, D, page, dtype, lens, tree=False, ragged=False, gate=None, seed=0, scale=None, q_std=1.0):
    pg = Paged(C, N, Hq, Hkv, D, page, dtype, lens, seed=seed)
    q = pg.normal(C, N, Hq, D, std=q_std)
    parents = random_parents(pg.rng, C, N) if tree else None
    nodes = pg.rng.integers(0, N + 1, C).astype(np.int32) if ragged else None
    z = None if gate is None else pg.normal(C, N, Hq, D)
    log(f"[attn] C={C} N={N} Hq={Hq} Hkv={Hkv} D={D} page={page} {dtype} lens={lens} tree={tree} ragged={ragged} gate={gate}")
    out, res, status, bits = _run(pg, q, parents, nodes, z, gate or 0, scale)
    assert status == bits == 0
    worst = check_attention(out, res, dtype, gate is not None)
    log(f"[attn]   worst error {worst:.3f} of the tolerance")


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_decode(dtype, D, G):
    _case(3, 1, 2 * G, 2, D, 16, dtype, [1, 70, 333], seed=G)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("N", [1, 2, 17, 32])
def test_trees(dtype, N):
    _case(3, N, 8, 2, 128, 48, dtype, [0, 65, 200], tree=True, ragged=N > 2, seed=N)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 256])
def test_chains_and_gate(dtype, D):
    for mode in (0, 1):
        _case(2, 9, 6, 2, D, 20, dtype, [63, 64], ragged=mode == 0, gate=mode, seed=mode)


@pytest.mark.parametrize("page", [1, 7, 16, 64, 100, 1000])
def test_page_sizes(page):
    _case(2, 5, 4, 2, 64, page, BF, [127, 129], seed=page)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("N,length", [(1, 0), (63, 0), (64, 1), (65, 64), (130, 37), (300, 0)])
def test_prompt_chunks(dtype, N, length):
    _case(1, N, 4, 2, 128, 64, dtype, [length], seed=N)


def test_many_row_tiles_share_a_head():
    _case(2, 257, 8, 1, 64, 32, BF, [5, 300], ragged=True, seed=3)


def test_long_cache_is_split_and_joined():
    _case(1, 1, 8, 2, 128, 64, BF, [5000], seed=1)
    _case(2, 3, 4, 4, 64, 16, FP, [4097, 31], seed=2)
    _case(1, 16, 16, 2, 256, 128, HF, [2500], tree=True, seed=4)


def test_sharp_scores_and_scale():
    _case(1, 4, 4, 2, 64, 16, BF, [200], q_std=30.0, seed=5)
    _case(1, 4, 4, 2, 64, 16, FP, [200], scale=3.0, seed=6)
    _case(1, 4, 4, 2, 64, 16, FP, [200], scale=1e-6, seed=7)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("tree", [False, True])
def test_rows_that_are_not_attended_may_hold_anything(dtype, bad, tree):
    """Non-finite keys and values behind the last token, in later tokens of the chain and in other branches."""
    C, N, page, lens = 2, 8, 16, [60, 3]
    pg = Paged(C, N, 4, 2, 64, page, dtype, lens, seed=11)
    q = pg.normal(C, N, 4, 64)
    parents = np.array([[-1, 0, 0, 1, 1, 2, -1, 6]] * C, np.int32) if tree else None
    clean = _run(pg, q, parents)[1]
    poisoned = 2  # the node whose row is poisoned: those that attend to it are left out of the comparison
    for c in range(C):
        s, n = int(pg.slots[c]), lens[c]
        for t in (n + poisoned, *range(n + N, pg.table.shape[1] * page)):
            pid = int(pg.table[s, t // page])
            if pid >= 0:
                pg.k[pid, :, t % page] = bad
                pg.v[pid, :, t % page] = bad
    spare = sorted(set(range(pg.sh.n_pages)) - set(pg.table[pg.table >= 0].tolist()))
    pg.k[spare], pg.v[spare] = bad, bad
    out = torch.full((C, N, 4, 64), SENTINEL, dtype=dtype, device="cuda")
    gdn.paged_attention(pg.sh, q, pg.k, pg.v, *pg.places(), parents=None if parents is None else dev(parents), out=out)
    seen = [i for i in range(N) if poisoned in R.path_of(None if parents is None else parents[0], i)]
    keep = [i for i in range(N) if i not in seen]
    got = as_numpy(out)
    assert not np.isfinite(got[:, seen]).any()
    for i in keep:
        for c in range(C):
            check_attention(out[c:c + 1, i:i + 1], {(0, 0): clean[c, i]}, dtype, ctx=f"node {i}")


def test_a_value_that_is_infinite_stays_with_its_readers():
    """An infinite value (finite key) of one column reaches exactly the nodes that attend to it, in that column."""
    pg = Paged(1, 6, 2, 1, 64, 32, BF, [40], seed=12)
    q = pg.normal(1, 6, 2, 64)
    clean, res, _, _ = _run(pg, q)
    pid = int(pg.table[pg.slots[0], (40 + 3) // 32])
    pg.v[pid, 0, (40 + 3) % 32, 17] = float("inf")
    out = as_numpy(_run(pg, q)[0])
    assert np.isposinf(out[0, 3:, :, 17]).all()
    out[0, 3:, :, 17] = as_numpy(clean)[0, 3:, :, 17]
    assert np.array_equal(out, as_numpy(clean))


def test_padding_invalid_lanes_and_bits():
    """Padding lanes and each kind of offending lane keep their output rows; the other lanes are computed."""
    C, N, page = 7, 4, 16
    pg = Paged(C, N, 4, 2, 64, page, BF, [30] * C, seed=13)
    q = pg.normal(C, N, 4, 64)
    slots, length = pg.slots.copy(), pg.len.copy()
    parents = random_parents(pg.rng, C, N)
    nodes = np.full(C, N, np.int32)
    slots[1] = -1
    slots[2] = pg.sh.n_slots
    nodes[3] = N + 1
    parents[4, 2] = 2
    length[slots[5]] = pg.sh.max_pages * page - N + 1
    out, res, status, bits = _run(pg, q, parents, nodes, slots=slots, length=length)
    assert status == bits == R.SLOT_RANGE | R.NODES | R.PARENT | R.LENGTH
    assert {c for c, _ in res} == {0, 6}
    check_attention(out, res, BF)
    slots[2:6] = -1  # padding only: no bits
    out, res, status, bits = _run(pg, q, parents, nodes, slots=slots, length=length)
    assert status == bits == 0
    check_attention(out, res, BF)
    length[slots[0]] = -1
    assert _run(pg, q, parents, nodes, slots=slots, length=length)[2] == R.LENGTH


@pytest.mark.parametrize("lens", [[30], [700]])
def test_rows_of_pages_outside_the_pool_are_not_attended(lens):
    pg = Paged(1, 3, 4, 2, 64, 16, BF, lens, seed=14)
    q = pg.normal(1, 3, 4, 64)
    table = pg.table.copy()
    for bad in (-7, pg.sh.n_pages, 2 ** 31 - 1, -2):
        table[pg.slots[0], 1] = bad
        out, res, status, bits = _run(pg, q, table=table)
        assert status == bits == R.PAGE
        check_attention(out, res, BF)
    table[pg.slots[0]] = -1  # nothing left to attend to
    out, _, status, _ = _run(pg, q, table=table)
    assert status == R.PAGE and (as_numpy(out) == 0).all()


def test_shared_slot_and_views():
    """Two lanes may read one slot; the gate may be a slice of a stacked projection."""
    pg = Paged(2, 2, 4, 2, 64, 16, BF, [50, 20], seed=15)
    q = pg.normal(2, 2, 4, 64)
    stacked = pg.normal(2, 2, 4, 128)
    out, res, status, bits = _run(pg, q, slots=np.array([pg.slots[0]] * 2, np.int32), gate=stacked[..., 64:], gate_mode=1)
    assert status == bits == 0
    check_attention(out, res, BF, gated=True)
    per_head = pg.normal(2, 2, 1, 64).expand(2, 2, 4, 64)  # one gate for all heads: a stride of zero
    out, res, _, _ = _run(pg, q, gate=per_head, gate_mode=0)
    check_attention(out, res, BF, gated=True)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes: its last pages are read where they lie."""
    page, D, Hkv = 128, 256, 4
    per = Hkv * page * D * 2
    n_pages = (1 << 32) // per + 40
    sh = gdn.AttnShape(1, 2, 1, 4, Hkv, D, page, n_pages, 3, BF)
    rng = np.random.default_rng(16)
    ids = [n_pages - 1, 3, n_pages - 17]
    small = Paged(1, 2, 4, Hkv, D, page, BF, [300], seed=17)
    k, v = (torch.zeros(sh.cache_shape, dtype=BF, device="cuda") for _ in range(2))
    for j, pid in enumerate(ids):
        src = int(small.table[small.slots[0], j])
        k[pid], v[pid] = small.k[src], small.v[src]
    q = dev(rng.standard_normal((1, 2, 4, D)).astype(np.float32), BF)
    want, _, _, _ = _run(small, q)
    ws = torch.empty(max(1, gdn.paged_attention_workspace_size(sh) // 4), device="cuda")
    got, status = gdn.paged_attention(sh, q, k, v, dev(np.zeros(1, np.int32)), dev(np.array([ids], np.int32)),
                                      dev(np.array([300], np.int32)), workspace=ws)
    assert int(status.item()) == 0 and torch.equal(got, want)


def test_results_do_not_change_between_runs_or_streams():
    pg = Paged(4, 16, 16, 4, 128, 64, BF, [900, 3, 2000, 64], seed=18)
    q = pg.normal(4, 16, 16, 128)
    parents = random_parents(pg.rng, 4, 16)
    first = _run(pg, q, parents)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = _run(pg, q, parents)[0]
    torch.cuda.synchronize()
    assert torch.equal(first, second)


def test_graph_replay_follows_lengths_and_inputs():
    """One captured call replayed with other lengths, pages and queries in the same buffers."""
    pg = Paged(2, 1, 8, 2, 128, 16, BF, [1500, 800], seed=19)
    q = pg.normal(2, 1, 8, 128)
    slots, table, length = pg.places()
    out = torch.zeros(2, 1, 8, 128, dtype=BF, device="cuda")
    ws = torch.empty(gdn.paged_attention_workspace_size(pg.sh) // 4, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: gdn.paged_attention(pg.sh, q, pg.k, pg.v, slots, table, length, out=out, workspace=ws, status=status)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(4):
        lens = [int(v) for v in pg.rng.integers(0, 1500, 2)]
        for c in range(2):
            pg.len[pg.slots[c]] = min(lens[c], 800 if c else 1500)
        length.copy_(dev(pg.len))
        q.copy_(pg.normal(2, 1, 8, 128))
        want = _run(pg, q)[0]
        out.zero_()
        ws.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {k}"
    assert int(status.item()) == 0


# Head layouts that reach every kernel: few rows, 64, 128 and 256 rows a workgroup, pairs of waves, each type
KERNELS = [(64, 2), (64, 8), (64, 16), (64, 40), (128, 2), (128, 8), (128, 16), (128, 40), (256, 1), (256, 2), (256, 40)]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
@pytest.mark.parametrize("tree", [False, True])
def test_poisoned_rows_in_every_kernel(dtype, D, G, tree):
    """As above, with a cache of several tiles, lanes of different lengths and a part that ends inside a tile: the
    nodes that attend to a poisoned row are not finite, the others are what they are without it."""
    C, N, page, lens = 2, 8, 48, [150, 61]
    pg = Paged(C, N, G, 1, D, page, dtype, lens, seed=D + G)
    q = pg.normal(C, N, G, D)
    parents = np.array([[-1, 0, 0, 1, 1, 2, -1, 6]] * C, np.int32) if tree else None
    clean, res, status, bits = _run(pg, q, parents)
    assert status == bits == 0
    check_attention(clean, res, dtype)
    poisoned = 2
    for c in range(C):
        s, n = int(pg.slots[c]), lens[c]
        for t in (n + poisoned, *range(n + N, pg.table.shape[1] * page)):
            pid = int(pg.table[s, t // page])
            if pid >= 0:
                pg.k[pid, :, t % page] = float("nan")
                pg.v[pid, :, t % page] = float("-inf") if c else float("nan")
    out = torch.full((C, N, G, D), SENTINEL, dtype=dtype, device="cuda")
    gdn.paged_attention(pg.sh, q, pg.k, pg.v, *pg.places(), parents=None if parents is None else dev(parents), out=out)
    seen = [i for i in range(N) if poisoned in R.path_of(None if parents is None else parents[0], i)]
    keep = [i for i in range(N) if i not in seen]
    got = as_numpy(out)
    assert not np.isfinite(got[:, seen]).any()
    assert np.array_equal(got[:, keep], as_numpy(clean)[:, keep])


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
def test_infinite_values_in_every_kernel(dtype, D, G):
    """Infinite values (finite keys) of the chain's own rows reach exactly the nodes that attend to them, in their
    column and with their sign, and NaN where both signs meet."""
    N, L = 6, 100
    pg = Paged(1, N, G, 1, D, 32, dtype, [L], seed=3 * D + G)
    q = pg.normal(1, N, G, D)
    clean = as_numpy(_run(pg, q)[0])

    def put(node, col, value):
        pg.v[int(pg.table[pg.slots[0], (L + node) // 32]), 0, (L + node) % 32, col] = value

    put(1, 3, float("inf"))
    put(3, D - 1, float("-inf"))
    put(2, 17, float("inf"))
    put(4, 17, float("-inf"))
    got = as_numpy(_run(pg, q)[0]).copy()
    assert np.isposinf(got[0, 1:, :, 3]).all() and np.isneginf(got[0, 3:, :, D - 1]).all()
    assert np.isposinf(got[0, 2:4, :, 17]).all() and np.isnan(got[0, 4:, :, 17]).all()
    for i, col in ((1, 3), (3, D - 1), (2, 17)):
        got[0, i:, :, col] = clean[0, i:, :, col]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_behind_long_caches(dtype, D):
    """Row tiles of every width over caches of many tiles, ragged and padded, with a gate."""
    _case(3, 70, 6, 2, D, 48, dtype, [700, 0, 321], ragged=True, gate=1, seed=D)
    _case(1, 33, 8, 1, D, 64, dtype, [1500], seed=D + 1)
    _case(2, 3, 12, 2, D, 16, dtype, [2000, 1], seed=D + 2)


@pytest.mark.parametrize("D,G,N", [(64, 4, 3), (64, 8, 8), (128, 16, 8), (128, 40, 8), (256, 2, 8), (256, 40, 8)])
def test_absent_pages_in_every_kernel(D, G, N):
    """Pages outside the pool in the first, a middle and the last place: their rows count as not attended to."""
    pg = Paged(2, N, G, 1, D, 16, BF, [200, 700], seed=D + G + 1)
    q = pg.normal(2, N, G, D)
    for at in (0, 5, (200 + N - 1) // 16):
        table = pg.table.copy()
        table[pg.slots[0], at] = pg.sh.n_pages + 3
        out, res, status, bits = _run(pg, q, table=table)
        assert status == R.PAGE and bits == R.PAGE
        check_attention(out, res, BF, ctx=f"page {at}")


@pytest.mark.parametrize("dtype,D,G", [(BF, 64, 2), (HF, 128, 1), (BF, 256, 1), (FP, 64, 1)])
def test_the_longest_chunk(dtype, D, G):
    """65536 tokens in one call, behind 77 rows: sampled rows, each as a single token behind those before it."""
    N, L = 65536, 77
    pg = Paged(1, N, G, 1, D, 256, dtype, [L], seed=D + G)
    q = pg.normal(1, N, G, D)
    out = torch.full((1, N, G, D), SENTINEL, dtype=dtype, device="cuda")
    ws = torch.empty(max(gdn.paged_attention_workspace_size(pg.sh) // 4, 1), device="cuda")
    _, status = gdn.paged_attention(pg.sh, q, pg.k, pg.v, *pg.places(), out=out, workspace=ws)
    assert int(status.item()) == 0
    k, v = as_numpy(pg.k), as_numpy(pg.v)
    for i in (0, 1, 127, 255, 256, 5000, 32767, 40001, 65279, 65534, 65535):
        length = np.where(np.arange(pg.sh.n_slots) == pg.slots[0], L + i, 0).astype(np.int32)
        res, bits = R.paged_attention(as_numpy(q[:, i:i + 1]), k, v, pg.slots, pg.table, length)
        assert bits == 0
        check_attention(out[:, i:i + 1], res, dtype, ctx=f"token {i}")


@pytest.mark.parametrize("dtype,D,N", [(BF, 128, 1), (FP, 256, 1), (HF, 256, 5), (FP, 64, 6)])
def test_the_most_lanes(dtype, D, N):
    """1024 lanes of every length from 0 to 60, some of them padding, shorter or sharing a page of the prefix."""
    C = 1024
    pg = Paged(C, N, 4, 1, D, 16, dtype, [c % 61 for c in range(C)], seed=D + N)
    slots, nodes = pg.slots.copy(), pg.rng.integers(0, N + 1, C).astype(np.int32)
    slots[::7] = -1
    for c in range(20, 1024, 61):  # lanes of 20 rows and more: the first page is full
        pg.table[pg.slots[c], 0] = pg.table[pg.slots[20], 0]
    out, res, status, bits = _run(pg, pg.normal(C, N, 4, D), None, nodes, slots=slots)
    assert status == bits == 0
    check_attention(out, res, dtype)


@pytest.mark.parametrize("dtype,N", [(FP, 6), (BF, 17), (HF, 17)])
def test_more_workgroups_than_a_round_with_the_cache_split(dtype, N):
    """260 groups of rows, two or three parts each, most of them behind a lane's last row."""
    C = 65
    pg = Paged(C, N, 16, 4, 64, 32, dtype, [(37 * c) % 601 for c in range(C)], seed=N)
    pg.table = np.pad(pg.table, ((0, 0), (0, 160 - pg.table.shape[1])), constant_values=-1)
    pg.sh = pg.sh._replace(max_pages=160)
    nodes = pg.rng.integers(0, N + 1, C).astype(np.int32)
    assert gdn.paged_attention_workspace_size(pg.sh) > 0
    out, res, status, bits = _run(pg, pg.normal(C, N, 16, 64), random_parents(pg.rng, C, N), nodes)
    assert status == bits == 0
    check_attention(out, res, dtype)
