"""The calls over a 4-bit cache against the fp64 oracle: attention (types, head layouts, page sizes, lengths from one token,
ragged and padded lanes, draft trees, gates, NaN blocks in rows that a node does not attend to), the quantising write, the
commit, rows read back, and a round of them together."""

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gpu_util import log
from kv4_util import Paged4
from oracle import kv4_oracle as K
from oracle import round_oracle as R
from round_util import HALF_STEP, SENTINEL, as_numpy, check_attention, dev, random_parents

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def _opt(a):
    return None if a is None else dev(a)


# ---------------------------------------------------------------- attention
def _run(pg, q, parents=None, lane_nodes=None, gate=None, gate_mode=1, scale=None, slots=None, table=None, length=None):
    sh = pg.sh
    out = torch.full((sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim), SENTINEL, dtype=sh.dtype, device="cuda")
    ws = torch.full((max(gdn.paged_attention_kv4_workspace_size(sh) // 4, 1),), float("nan"), device="cuda")
    s, t, n = (pg.slots if slots is None else slots, pg.table if table is None else table, pg.len if length is None else length)
    _, status = gdn.paged_attention_kv4(sh, q, pg.cache, dev(s), dev(t), dev(n), parents=_opt(parents),
                                        lane_nodes=_opt(lane_nodes), gate=gate, gate_mode=gate_mode, scale=scale, out=out,
                                        workspace=ws)
    torch.cuda.synchronize()
    res, bits = R.paged_attention(as_numpy(q), *pg.values(), s, t, n, parents, lane_nodes, scale,
                                  None if gate is None else as_numpy(gate), gate_mode)
    return out, res, int(status.item()), bits


def _case(C, N, Hq, Hkv, D, page, dtype, lens, tree=False, ragged=False, gate=None, seed=0, scale=None, q_std=1.0):
    pg = Paged4(C, N, Hq, Hkv, D, page, dtype, lens, seed=seed)
    q = pg.normal(C, N, Hq, D, std=q_std)
    parents = random_parents(pg.rng, C, N) if tree else None
    nodes = pg.rng.integers(0, N + 1, C).astype(np.int32) if ragged else None
    z = None if gate is None else pg.normal(C, N, Hq, D)
    log(f"[kv4] C={C} N={N} Hq={Hq} Hkv={Hkv} D={D} page={page} {dtype} lens={lens} tree={tree} ragged={ragged} gate={gate}")
    out, res, status, bits = _run(pg, q, parents, nodes, z, gate or 0, scale)
    assert status == bits == 0
    worst = check_attention(out, res, dtype, gate is not None)
    log(f"[kv4]   worst error {worst:.3f} of the tolerance")


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 3, 8])
def test_decode(dtype, D, G):
    _case(3, 1, 2 * G, 2, D, 16, dtype, [1, 70, 333], seed=G)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,N", [(128, 1), (128, 2), (64, 17), (128, 17), (256, 17), (64, 32), (128, 32), (256, 32)])
def test_trees(dtype, D, N):
    _case(3, N, 8, 2, D, 48, dtype, [0, 65, 200], tree=True, ragged=N > 2, seed=N)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("D", [64, 256])
def test_chains_and_gate(dtype, D):
    for mode in (0, 1):
        _case(2, 9, 6, 2, D, 20, dtype, [63, 64], ragged=mode == 0, gate=mode, seed=mode)


@pytest.mark.parametrize("page", [1, 7, 16, 64, 100, 1000])
def test_page_sizes(page):
    _case(2, 5, 4, 2, 64, page, BF, [127, 129], seed=page)


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N,length", [(1, 0), (63, 0), (64, 1), (65, 64), (130, 37), (300, 0)])
def test_prompt_chunks(dtype, D, N, length):
    _case(1, N, 4, 2, D, 64, dtype, [length], seed=N)


def test_long_cache_is_split_and_joined():
    _case(1, 1, 8, 2, 128, 64, BF, [5000], seed=1)
    _case(2, 3, 4, 4, 64, 16, FP, [4097, 31], seed=2)
    _case(1, 16, 16, 2, 256, 128, HF, [2500], tree=True, seed=4)
    _case(1, 1, 4, 1, 256, 128, FP, [3001], seed=5)


def test_sharp_scores_and_scale():
    _case(1, 4, 4, 2, 64, 16, BF, [200], q_std=30.0, seed=5)
    _case(1, 4, 4, 2, 64, 16, FP, [200], scale=3.0, seed=6)
    _case(1, 4, 4, 2, 64, 16, FP, [200], scale=1e-6, seed=7)


# Head layouts that reach every kernel: few rows, 64, 128 and 256 rows a workgroup, pairs of waves, each type
KERNELS = [(64, 2), (64, 8), (64, 16), (64, 40), (128, 2), (128, 8), (128, 16), (128, 40), (256, 1), (256, 2), (256, 40)]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
@pytest.mark.parametrize("tree", [False, True])
def test_nan_blocks_of_rows_that_are_not_attended(dtype, D, G, tree):
    """NaN blocks behind the last token, in later tokens of the chain and in other branches: the nodes that attend to
    one are not finite, the others are what they are without it."""
    C, N, page, lens = 2, 8, 48, [150, 61]
    pg = Paged4(C, N, G, 1, D, page, dtype, lens, seed=D + G)
    q = pg.normal(C, N, G, D)
    parents = np.array([[-1, 0, 0, 1, 1, 2, -1, 6]] * C, np.int32) if tree else None
    clean, res, status, bits = _run(pg, q, parents)
    assert status == bits == 0
    check_attention(clean, res, dtype)
    poisoned = 2
    for c in range(C):
        for t in (lens[c] + poisoned, *range(lens[c] + N, pg.table.shape[1] * page)):
            if pg.table[pg.slots[c], t // page] >= 0:
                pid, at = pg.place(c, t)
                pg.cache.k_scale[pid, :, at] = 255
                pg.cache.v_scale[pid, :, at] = 255
    spare = sorted(set(range(pg.sh.n_pages)) - set(pg.table[pg.table >= 0].tolist()))
    pg.cache.k_scale[spare], pg.cache.v_scale[spare] = 255, 255
    out = torch.full((C, N, G, D), SENTINEL, dtype=dtype, device="cuda")
    gdn.paged_attention_kv4(pg.sh, q, pg.cache, *pg.places(), parents=_opt(parents), out=out)
    seen = [i for i in range(N) if poisoned in R.path_of(None if parents is None else parents[0], i)]
    keep = [i for i in range(N) if i not in seen]
    got = as_numpy(out)
    assert not np.isfinite(got[:, seen]).any()
    assert np.array_equal(got[:, keep], as_numpy(clean)[:, keep])


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,G", KERNELS)
def test_a_nan_value_block_stays_in_its_columns(dtype, D, G):
    """A value block of scale 255 in the chain makes its 32 columns NaN for the nodes that attend to the row."""
    N, L = 6, 100
    pg = Paged4(1, N, G, 1, D, 32, dtype, [L], seed=3 * D + G)
    q = pg.normal(1, N, G, D)
    clean = as_numpy(_run(pg, q)[0])
    pid, at = pg.place(0, L + 3)
    pg.cache.v_scale[pid, 0, at, 1] = 255
    out = torch.empty(1, N, G, D, dtype=dtype, device="cuda")
    gdn.paged_attention_kv4(pg.sh, q, pg.cache, *pg.places(), out=out)
    got = as_numpy(out).copy()
    assert np.isnan(got[0, 3:, :, 32:64]).all()
    got[0, 3:, :, 32:64] = clean[0, 3:, :, 32:64]
    assert np.array_equal(got, clean)


@pytest.mark.parametrize("dtype", [BF, FP, HF])
@pytest.mark.parametrize("D,N", [(64, 1), (128, 1), (256, 1), (128, 40), (256, 40)])
def test_scales_at_the_ends_of_the_range(dtype, D, N):
    """Blocks of very small and very large powers of two: keys cancel the queries' sizes, values keep theirs."""
    pg = Paged4(1, N, 4, 1, D, 16, dtype, [60], seed=N + D)
    low, high = (120, 140) if dtype is HF else (2, 200)
    q = pg.normal(1, N, 4, D, std=2.0 ** -9 if dtype is HF else 2.0 ** -70)
    pg.host[1][:] = 127 + (8 if dtype is HF else 70)
    pg.host[3][...] = np.where(np.arange(D // 32) % 2, low, high)
    pg.push()
    out, res, status, bits = _run(pg, q)
    assert status == bits == 0
    check_attention(out, res, dtype)


def test_padding_invalid_lanes_and_bits():
    C, N, page = 7, 4, 16
    pg = Paged4(C, N, 4, 2, 64, page, BF, [30] * C, seed=13)
    q = pg.normal(C, N, 4, 64)
    slots, length = pg.slots.copy(), pg.len.copy()
    parents, nodes = random_parents(pg.rng, C, N), np.full(C, N, np.int32)
    slots[1] = -1
    slots[2] = pg.sh.n_slots
    nodes[3] = N + 1
    parents[4, 2] = 2
    length[slots[5]] = pg.sh.max_pages * page - N + 1
    out, res, status, bits = _run(pg, q, parents, nodes, slots=slots, length=length)
    assert status == bits == R.SLOT_RANGE | R.NODES | R.PARENT | R.LENGTH
    assert {c for c, _ in res} == {0, 6}
    check_attention(out, res, BF)


@pytest.mark.parametrize("D,G,N", [(64, 4, 3), (64, 8, 8), (128, 16, 8), (128, 40, 8), (256, 2, 8), (256, 40, 8)])
def test_absent_pages_in_every_kernel(D, G, N):
    """Pages outside the pool in the first, a middle and the last place: their rows count as not attended to."""
    pg = Paged4(2, N, G, 1, D, 16, BF, [200, 700], seed=D + G + 1)
    q = pg.normal(2, N, G, D)
    for at, bad in ((0, -7), (5, pg.sh.n_pages), ((200 + N - 1) // 16, 2 ** 31 - 1)):
        table = pg.table.copy()
        table[pg.slots[0], at] = bad
        out, res, status, bits = _run(pg, q, table=table)
        assert status == R.PAGE and bits == R.PAGE
        check_attention(out, res, BF, ctx=f"page {at}")
    table[pg.slots[0]] = -1  # nothing left to attend to
    out, _, status, _ = _run(pg, q, table=table)
    assert status == R.PAGE and (as_numpy(out)[0] == 0).all()


def test_shared_slot_views_and_streams():
    """Two lanes may read one slot; the gate may be a slice of a stacked projection; another stream gives the same bits."""
    pg = Paged4(2, 2, 4, 2, 64, 16, BF, [50, 20], seed=15)
    q = pg.normal(2, 2, 4, 64)
    stacked = pg.normal(2, 2, 4, 128)
    shared = np.array([pg.slots[0]] * 2, np.int32)
    out, res, status, bits = _run(pg, q, slots=shared, gate=stacked[..., 64:], gate_mode=1)
    assert status == bits == 0
    check_attention(out, res, BF, gated=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _run(pg, q, slots=shared, gate=stacked[..., 64:], gate_mode=1)[0]
    torch.cuda.synchronize()
    assert torch.equal(out, again)


def test_offsets_past_32_bits():
    """A pool whose codes fill more than 2^32 bytes: its last pages are read, written and moved where they lie."""
    page, D, Hkv, N, L = 128, 256, 8, 6, 250
    n_pages = (1 << 32) // (Hkv * page * D // 2) + 40
    ids = np.array([[n_pages - 1, n_pages - 17]], np.int32)
    small = Paged4(1, N, 16, Hkv, D, page, BF, [L], seed=17, extra_slots=0)
    sh = small.sh._replace(n_pages=n_pages)
    big = gdn.kv4_cache(sh)
    for b, s in zip(big, small.cache):
        for j in range(2):
            b[int(ids[0, j])] = s[int(small.table[0, j])]
    x = small.normal(1, N, 16 + 2 * Hkv, D)
    inv, (slots, table, length) = dev(1e4 ** (-np.arange(64) / 64)), small.places()
    parents, accept = dev(np.array([[-1, 0, 0, 1, 2, 3]], np.int32)), dev(np.array([5], np.int32))
    outs = []
    for s, cache, tab in ((small.sh, small.cache, table), (sh, big, dev(ids))):
        q, status = gdn.rope_kv4_write(s, x[:, :, :16], x[:, :, 16:16 + Hkv], x[:, :, 16 + Hkv:], inv, cache, slots, tab, length,
                                       parents=parents)
        out, _ = gdn.paged_attention_kv4(s, q, cache, slots, tab, length, parents=parents, status=status)
        gdn.kv4_commit_layers(s, [cache], slots, tab, length, accept, status, parents=parents)
        k, v, _ = gdn.kv4_read_layers(s, [cache], slots, tab, dev(np.array([L - 2], np.int32)), status=status)
        assert int(status.item()) == 0
        outs.append((out, k, v))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    for b, s in zip(big, small.cache):
        for j in range(2):
            assert torch.equal(b[int(ids[0, j])], s[int(small.table[0, j])])


def test_graph_replay_follows_lengths_and_inputs():
    pg = Paged4(2, 1, 8, 2, 128, 16, BF, [1500, 800], seed=19)
    q = pg.normal(2, 1, 8, 128)
    slots, table, length = pg.places()
    out = torch.zeros(2, 1, 8, 128, dtype=BF, device="cuda")
    ws = torch.empty(max(1, gdn.paged_attention_kv4_workspace_size(pg.sh) // 4), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: gdn.paged_attention_kv4(pg.sh, q, pg.cache, slots, table, length, out=out, workspace=ws, status=status)  # noqa: E731
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(4):
        for c in range(2):
            pg.len[pg.slots[c]] = int(pg.rng.integers(0, 800 if c else 1500))
        length.copy_(dev(pg.len))
        q.copy_(pg.normal(2, 1, 8, 128))
        want = _run(pg, q)[0]
        out.zero_()
        ws.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), f"replay {k}"
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype,D,N", [(BF, 128, 1), (FP, 256, 1), (HF, 256, 5), (FP, 64, 6)])
def test_the_most_lanes(dtype, D, N):
    C = 1024
    pg = Paged4(C, N, 4, 1, D, 16, dtype, [c % 61 for c in range(C)], seed=D + N)
    slots, nodes = pg.slots.copy(), pg.rng.integers(0, N + 1, C).astype(np.int32)
    slots[::7] = -1
    out, res, status, bits = _run(pg, pg.normal(C, N, 4, D), None, nodes, slots=slots)
    assert status == bits == 0
    check_attention(out, res, dtype)


@pytest.mark.parametrize("dtype,D", [(BF, 64), (BF, 128), (HF, 256), (FP, 128)])
def test_chunks_behind_long_caches(dtype, D):
    _case(3, 70, 6, 2, D, 48, dtype, [700, 0, 321], ragged=True, gate=1, seed=D)
    _case(1, 33, 8, 1, D, 64, dtype, [1500], seed=D + 1)
    _case(2, 3, 12, 2, D, 16, dtype, [2000, 1], seed=D + 2)


@pytest.mark.parametrize("dtype,D,G", [(BF, 64, 2), (BF, 256, 1)])
def test_the_longest_chunk(dtype, D, G):
    """65536 tokens in one call, behind 77 rows: sampled rows, each as a single token behind those before it."""
    N, L = 65536, 77
    pg = Paged4(1, N, G, 1, D, 256, dtype, [L], seed=D + G)
    q = pg.normal(1, N, G, D)
    out, status = gdn.paged_attention_kv4(pg.sh, q, pg.cache, *pg.places())
    assert int(status.item()) == 0
    values = pg.values()
    for i in (0, 1, 127, 255, 256, 5000, 32767, 40001, 65279, 65534, 65535):
        length = np.where(np.arange(pg.sh.n_slots) == pg.slots[0], L + i, 0).astype(np.int32)
        res, bits = R.paged_attention(as_numpy(q[:, i:i + 1]), *values, pg.slots, pg.table, length)
        assert bits == 0
        check_attention(out[:, i:i + 1], res, dtype, ctx=f"token {i}")


# ---------------------------------------------------------------- the quantising write
def _write(pg, q, k, v, half, parents=None, nodes=None, slots=None, length=None, table=None, **kw):
    """Every row that the oracle writes lies on the grid of its block and no further from the exact value than the
    nearest grid point and the value's own error; every other byte is as it was.  Returns the status."""
    sh = pg.sh
    inv = 1e4 ** (-np.arange(half) / half)
    q_out = torch.full((sh.n_seqs, sh.n_nodes, sh.n_q_heads, sh.head_dim), SENTINEL, dtype=sh.dtype, device="cuda")
    s, t, n = (pg.slots if slots is None else slots, pg.table if table is None else table, pg.len if length is None else length)
    before = pg.pull()
    gpu = {a: _opt(b) if isinstance(b, np.ndarray) else b for a, b in kw.items()}
    _, status = gdn.rope_kv4_write(sh, q, k, v, dev(inv), pg.cache, dev(s), dev(t), dev(n), parents=_opt(parents),
                                   lane_nodes=_opt(nodes), q_out=q_out, **gpu)
    plain, _ = gdn.rope_kv_write(sh, q, k, v, dev(inv), *(torch.zeros(sh.cache_shape, dtype=sh.dtype, device="cuda") for _ in range(2)),
                                 dev(s), dev(t), dev(n), parents=_opt(parents), lane_nodes=_opt(nodes),
                                 q_out=torch.full_like(q_out, SENTINEL), **gpu)
    torch.cuda.synchronize()
    assert torch.equal(q_out, plain)  # the queries are those of the other cache's call
    pos = kw.get("positions")
    _, kx, vx, bits = K.rope_rows(as_numpy(q), as_numpy(k), as_numpy(v), inv, sh.n_kv_heads, sh.page_size, sh.n_pages, s, t, n,
                                  parents=parents, lane_nodes=nodes, n_axes=1 if pos is None else pos.shape[2], **kw)
    assert int(status.item()) == bits
    after = pg.pull()
    for x, j, turned in ((kx, 0, True), (vx, 2, False)):
        written = ~np.isnan(x).all(-1)
        for a, b in ((before[j], after[j]), (before[j + 1], after[j + 1])):
            assert np.array_equal(a[~written], b[~written]), "a row that is not the round's was written"
        rows, codes, scales = x[written], after[j][written], after[j + 1][written]
        got = K.values(codes, scales)
        for r in range(len(rows)):
            # a value's own error: as in the other cache's test (rotation and norm in 32 bits), none for v
            tol = np.sqrt((rows[r] ** 2).sum()) * (2.0 ** -19 + (sh.head_dim + 4) * 2.0 ** -24) if turned else 0.0
            for b in range(sh.head_dim // 32):
                blk = slice(32 * b, 32 * b + 32)
                a, most = float(np.abs(rows[r, blk]).max()), 13 if sh.dtype is HF else 125
                e = int(scales[r, b]) - 127
                assert K.exponent(max(a - tol, 0.0), most) <= e <= K.exponent(a + tol, most), (r, b, a, e)
                grid = 2.0 ** e * np.array(sorted({s * m for m in K.MAGNITUDES for s in (1, -1)}))
                off = np.abs(rows[r, blk, None] - grid).min(-1)
                assert (np.abs(got[r, blk] - rows[r, blk]) <= off + 2 * tol).all(), (r, b)
            if not turned:  # exact inputs: exactly the oracle's bytes
                want = K.quantise(rows[r], sh.dtype is HF)
                assert np.array_equal(codes[r], want[0]) and np.array_equal(scales[r], want[1])
    return bits


def _qkv(pg, xdtype):
    sh = pg.sh
    x = pg.normal(sh.n_seqs, sh.n_nodes, sh.n_q_heads + 2 * sh.n_kv_heads, sh.head_dim, dtype=xdtype)
    a, b = sh.n_q_heads, sh.n_q_heads + sh.n_kv_heads
    return x[:, :, :a], x[:, :, a:b], x[:, :, b:]


@pytest.mark.parametrize("xdtype,dtype", [(BF, BF), (HF, HF), (FP, FP), (FP, BF), (FP, HF)])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 16), (128, 128), (256, 64), (256, 240)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_write_types_and_widths(xdtype, dtype, D, rot, interleaved):
    pg = Paged4(2, 3, 6, 2, D, 16, dtype, [15, 40], seed=rot)
    assert _write(pg, *_qkv(pg, xdtype), rot // 2, interleaved=interleaved) == 0


@pytest.mark.parametrize("D", [64, 128, 256])
def test_write_axes_norms_trees_and_ragged_lanes(D):
    C, N = 3, 9
    pg = Paged4(C, N, 5, 1, D, 7, BF, [0, 33, 12], seed=D)
    half = D // 4
    w = lambda: (1 + 0.2 * pg.rng.standard_normal(D)).astype(np.float32)  # noqa: E731
    parents, nodes = random_parents(pg.rng, C, N), np.array([N, 0, 4], np.int32)
    q, k, v = _qkv(pg, FP)
    _write(pg, q, k, v, half, parents, nodes, q_norm=w(), k_norm=w(), eps=1e-5)
    _write(pg, q, k, v, half, q_norm=None, k_norm=w(), eps=1e-5)
    pos = pg.rng.integers(-5, 1 << 22, (C, N, 3)).astype(np.int32)
    _write(pg, q, k, v, half, positions=pos, pair_axis=(np.arange(half) % 3).astype(np.int32))


@pytest.mark.parametrize("xdtype,dtype", [(FP, FP), (FP, HF), (BF, BF), (HF, HF)])
def test_write_ties_borders_and_extremes(xdtype, dtype):
    """Values of v on the borders between two codes and two scales, zeros of both signs, the largest and the smallest."""
    D, N = 128, 8
    pg = Paged4(1, N, 1, 1, D, 16, dtype, [3], seed=2)
    q, k, v = (t.clone() for t in _qkv(pg, xdtype))
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1, 1.5, 2, 3, 4, 6, 0.0, -0.0])
    rows = np.zeros((N, D))
    for i, top in enumerate((6.0, 6.9375, 7.0, 7.03125, 3.5)):
        rows[i, :32] = np.concatenate((ties, -ties))
        rows[i, 5], rows[i, 21] = top, -min(top, 5.0)
        rows[i, 32:64] = rows[i, :32] * 2.0 ** -7
        rows[i, 64:96] = rows[i, :32] * 2.0 ** 6
    if dtype is HF:  # above 6 * 2^13 values are clipped; half's own smallest ones
        rows[5, :32], rows[5, 32:64], rows[5, 64:96] = 65504.0 * np.sign(rows[0, :32] - 0.1), 2.0 ** -14, 2.0 ** -20
    else:
        big = 3.3895313892515355e38  # bfloat16's largest
        rows[5, :32], rows[5, 32:64], rows[5, 64:96] = big * np.sign(rows[0, :32] - 0.1), 2.0 ** -100, -2.0 ** -126
    v[0, :, 0] = dev(rows.astype(np.float32), xdtype)
    assert np.array_equal(as_numpy(v[0, :, 0]), rows.astype(np.float32))  # (every one is a value of the type)
    assert _write(pg, q, k, v, 16) == 0


def test_write_of_nan_and_infinity_marks_their_blocks():
    pg = Paged4(1, 4, 2, 1, 64, 16, FP, [3], seed=2)
    q, k, v = (t.clone() for t in _qkv(pg, FP))
    clean = [t.clone() for t in (k, v)]
    k[0, 0, 0, 40], v[0, 1, 0, 3], v[0, 2, 0, 63], k[0, 3, 0, 50] = float("nan"), float("inf"), float("-inf"), float("inf")
    inv = dev(1e4 ** (-np.arange(8) / 8))  # values from 16 on keep their places
    out = []
    for kk, vv in ((k, v), clean):
        pg.push()
        gdn.rope_kv4_write(pg.sh, q, kk, vv, inv, pg.cache, *pg.places())
        out.append([as_numpy(t) for t in gdn.kv4_read_layers(pg.sh, [pg.cache], dev(pg.slots), dev(pg.table), dev(np.array([3], np.int32)))[:2]])
    (gk, gv), (ck, cv) = out
    for got, want, where in ((gk, ck, {(0, 1), (3, 1)}), (gv, cv, {(1, 0), (2, 1)})):
        for i in range(4):
            for b in range(2):
                g, w = got[0, 0, i, 0, 32 * b:32 * b + 32], want[0, 0, i, 0, 32 * b:32 * b + 32]
                assert np.isnan(g).all() if (i, b) in where else np.array_equal(g, w)


def test_write_refuses_lanes_and_pages():
    C, N = 6, 3
    pg = Paged4(C, N, 2, 1, 64, 4, BF, [6] * C, seed=4)
    slots, length, parents, nodes = pg.slots.copy(), pg.len.copy(), random_parents(pg.rng, C, N), np.full(C, N, np.int32)
    slots[1] = slots[0]
    slots[2] = -3
    nodes[3] = -1
    parents[4, 1] = 1
    q, k, v = _qkv(pg, BF)
    assert _write(pg, q, k, v, 16, parents, nodes, slots=slots) == R.SLOT_DUP | R.SLOT_RANGE | R.NODES | R.PARENT
    table = pg.table.copy()
    table[pg.slots[0], 2] = pg.sh.n_pages  # holds the last row of the round
    assert _write(pg, q, k, v, 16, table=table) == R.PAGE
    assert _write(pg, q, k, v, 16, positions=np.zeros((C, N, 2), np.int32), pair_axis=np.full(16, 2, np.int32)) == R.AXIS
    assert _write(pg, q, k, v, 16, slots=np.full(C, -1, np.int32)) == 0


# ---------------------------------------------------------------- commit and rows read back
def _commit(pg, accept, parents=None, nodes=None, slots=None, table=None, length=None, status_in=0, as_list=False):
    s, t, n = (pg.slots if slots is None else slots, pg.table if table is None else table, pg.len if length is None else length)
    before = pg.pull()
    status = torch.full((1,), status_in, dtype=torch.int32, device="cuda")
    caches = [gdn.Kv4Cache(*c) for c in zip(*pg.cache)] if as_list else pg.cache
    new_len = gdn.kv4_commit_layers(pg.sh, caches, dev(s), dev(t), dev(n), dev(np.asarray(accept, np.int32)), status,
                                    parents=_opt(parents), lane_nodes=_opt(nodes))
    torch.cuda.synchronize()
    layers = [a[l] for a in before for l in range(len(a))]  # copies to move rows in
    half = len(layers) // 2
    want_len, bits = R.kv_commit(layers[:half], layers[half:], s, t, n, accept, parents, nodes, status_in, N=pg.sh.n_nodes)
    assert int(status.item()) == bits and np.array_equal(as_numpy(new_len), want_len)
    for got, want in zip(pg.pull(), before):  # (moved in place above)
        assert np.array_equal(got, want)
    return bits


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("N", [1, 2, 7, 32])
def test_commit_moves_rows_of_every_layer(D, N):
    C = 4
    pg = Paged4(C, N, 3, 3, D, 5, BF, [0, 4, 33, 17], seed=N + D, layers=3)
    parents, nodes = random_parents(pg.rng, C, N), pg.rng.integers(1, N + 1, C).astype(np.int32)
    for as_list in (False, True):
        accept = np.minimum(pg.rng.integers(-1, N, C), nodes - 1).astype(np.int32)
        assert _commit(pg, accept, parents, nodes, as_list=as_list) == 0
    assert _commit(pg, np.full(C, N - 1), None) == 0  # a chain: lengths only
    chain = np.tile(np.arange(-1, N - 1, dtype=np.int32), (C, 1))
    assert _commit(pg, np.full(C, N - 1), chain) == 0


def test_commit_is_a_transaction():
    C, N = 4, 6
    pg = Paged4(C, N, 2, 1, 64, 8, BF, [20, 3, 9, 40], seed=9, layers=2)
    parents, accept = random_parents(pg.rng, C, N), np.array([5, 3, 0, 2], np.int32)
    assert _commit(pg, accept, parents, status_in=2) == 2
    slots, length, table, p = pg.slots.copy(), pg.len.copy(), pg.table.copy(), parents.copy()
    slots[3] = slots[0]
    assert _commit(pg, accept, parents, slots=slots) == R.SLOT_DUP
    p[3, 4] = 5
    assert _commit(pg, accept, p) == R.PARENT
    assert _commit(pg, np.array([5, 3, 6, 2]), parents) == R.ACCEPT
    length[pg.slots[0]] = pg.sh.max_pages * 8
    assert _commit(pg, accept, parents, length=length) == R.LENGTH
    table[pg.slots[1], 0] = -1
    assert _commit(pg, accept, parents, table=table) == R.PAGE


def test_commit_of_many_layers_and_lanes():
    C, N = 300, 4
    pg = Paged4(C, N, 2, 2, 64, 16, HF, [c % 37 for c in range(C)], seed=3, layers=64)
    assert _commit(pg, pg.rng.integers(-1, N, C).astype(np.int32), random_parents(pg.rng, C, N)) == 0


def _read(pg, first, nodes=None, slots=None, table=None, only=None, sh=None):
    sh = pg.sh if sh is None else sh
    s, t = pg.slots if slots is None else slots, pg.table if table is None else table
    n = len(pg.host[0])
    outs = [torch.full((n, sh.n_seqs, sh.n_nodes, sh.n_kv_heads, sh.head_dim), SENTINEL, dtype=sh.dtype, device="cuda") for _ in range(2)]
    _, _, status = gdn.kv4_read_layers(sh, pg.cache, dev(s), dev(t), dev(np.asarray(first, np.int32)), lane_nodes=_opt(nodes),
                                       k_out=outs[0], v_out=outs[1])
    torch.cuda.synchronize()
    bits = 0
    for got, j in zip(outs, (0, 2)):
        got = as_numpy(got)
        for l in range(n):
            want, b = K.read(pg.host[j][l], pg.host[j + 1][l], s, t, first, sh.n_nodes, nodes)
            bits |= b
            for c in range(sh.n_seqs):
                for i in range(sh.n_nodes):
                    w = want.get((c, i))
                    if w is None:
                        assert (got[l, c, i] == SENTINEL).all()
                    else:
                        w = torch.from_numpy(w).to(sh.dtype).float().numpy()
                        assert np.array_equal(got[l, c, i], w, equal_nan=True)
    assert int(status.item()) == bits
    return bits


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("D,Hkv,N", [(64, 1, 1), (64, 3, 40), (128, 2, 17), (256, 1, 33), (256, 5, 2)])
def test_read_rows(dtype, D, Hkv, N):
    pg = Paged4(3, N, Hkv, Hkv, D, 7, dtype, [0, 20, 44], seed=D + N, layers=2)
    for j in (1, 3):  # every scale, NaN blocks among them
        pg.host[j][:] = pg.rng.integers(0, 256, pg.host[j].shape)
    if dtype is BF:  # (2^128 and 1.5 * 2^128 have no value there)
        for j in (1, 3):
            pg.host[j][(pg.host[j] > 252) & (pg.host[j] < 255)] = 252
    if dtype is FP:
        for j in (1, 3):
            pg.host[j][(pg.host[j] > 252) & (pg.host[j] < 255)] = 252
    pg.push()
    assert _read(pg, [0, 20, 13]) == 0
    assert _read(pg, [0, 3, 40], nodes=pg.rng.integers(0, N + 1, 3).astype(np.int32)) == 0


def test_read_refuses_lanes_and_pages():
    C, N = 6, 3
    pg = Paged4(C, N, 2, 1, 64, 4, BF, [6] * C, seed=4, layers=1)
    slots, nodes, first = pg.slots.copy(), np.full(C, N, np.int32), np.full(C, 6, np.int32)
    slots[0], slots[1], nodes[2], first[3], first[4] = -1, pg.sh.n_slots, N + 1, -1, pg.sh.max_pages * 4 - 2
    assert _read(pg, first, nodes, slots=slots) == R.SLOT_RANGE | R.NODES | R.LENGTH
    table = pg.table.copy()
    table[pg.slots[0], 2] = -1
    assert _read(pg, np.full(C, 6), table=table) == R.PAGE
    assert _read(pg, np.full(C, 0), slots=np.full(C, pg.slots[2], np.int32)) == 0  # lanes share a slot


# ---------------------------------------------------------------- a round, as it is used
@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_rounds_over_a_4_bit_cache(graph, dtype):
    """Three rounds without host synchronisation: the quantising write, attention over the draft tree, greedy acceptance
    on the device and the commit by its accept_node; then the committed rows read back.  Each round's attention is
    held against the oracle on the bytes that the device holds at that time."""
    C, N, V, Hq, Hkv, D, page, rounds = 3, 12, 97, 4, 2, 64, 16, 3
    pg = Paged4(C, rounds * N, Hq, Hkv, D, page, dtype, [21, 0, 50], seed=7, layers=1)
    sh, rng = pg.sh._replace(n_nodes=N), pg.rng
    layer = gdn.Kv4Cache(*(t[0] for t in pg.cache))
    feed = []
    for r in range(rounds):
        parents = random_parents(rng, C, N)
        p = rng.standard_normal((C, N + 1, V)).astype(np.float32)
        tokens = np.empty((C, N), np.int32)
        for c in range(C):
            for i in range(N):
                tokens[c, i] = int(np.argmax(p[c, parents[c, i] + 1])) if rng.random() < 0.8 else rng.integers(V)
        feed.append(dict(parents=parents, target=p[:, 1:], root=p[:, 0], tokens=tokens,
                         x=rng.standard_normal((C, N, Hq + 2 * Hkv, D)).astype(np.float32)))
    buf = {k: dev(v) for k, v in feed[0].items()}
    slots, table, length = pg.places()
    l0, inv = length.clone(), dev(1e4 ** (-np.arange(32) / 32))
    new_len, status = torch.zeros_like(length), torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out, att = (torch.zeros(C, N, Hq, D, dtype=dtype, device="cuda") for _ in range(2))
    ws = torch.empty(max(1, gdn.paged_attention_kv4_workspace_size(sh) // 4), device="cuda")
    ash = gdn.AcceptShape(C, N, V, FP)
    aws = torch.empty(gdn.draft_accept_workspace_size(ash) // 4, device="cuda")
    acc = [torch.zeros(C, dtype=torch.int32, device="cuda") for _ in range(3)]
    held = gdn.Kv4Cache(*(torch.zeros_like(t) for t in pg.cache))

    def one_round():
        x = buf["x"]
        gdn.rope_kv4_write(sh, x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], inv, layer, slots, table, length,
                           parents=buf["parents"], q_out=q_out, status=status)
        gdn.paged_attention_kv4(sh, q_out, layer, slots, table, length, parents=buf["parents"], out=att, workspace=ws, status=status)
        for a, b in zip(held, pg.cache):
            a.copy_(b)
        gdn.draft_accept(ash, buf["target"], buf["tokens"], root_target=buf["root"], parents=buf["parents"], slot_ids=slots,
                         accept_node=acc[0], n_accept=acc[1], next_token=acc[2], workspace=aws, status=status)
        gdn.kv4_commit_layers(sh, pg.cache, slots, table, length, acc[0], status, parents=buf["parents"], new_len=new_len)
        length.copy_(new_len)

    replay = one_round
    if graph:
        one_round()  # warms up
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            one_round()
        length.copy_(l0)
        pg.push()
        replay = g.replay
    saved = []
    for r in range(rounds):
        for key, v in feed[r].items():
            buf[key].copy_(dev(v))
        replay()
        saved.append((q_out.clone(), att.clone(), [t.clone() for t in held], acc[0].clone(), length.clone(), [t.clone() for t in pg.cache]))
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    lens, moved = as_numpy(l0), 0
    for r, (q, out, bytes_, node, new, after) in enumerate(saved):
        host = [as_numpy(t)[0] for t in bytes_]
        k, v = K.values(host[0], host[1]), K.values(host[2], host[3])
        res, bits = R.paged_attention(as_numpy(q), k, v, pg.slots, pg.table, lens, parents=feed[r]["parents"])
        assert bits == 0
        check_attention(out, res, dtype, ctx=f"round {r}")
        got, _ = R.draft_accept(feed[r]["target"], feed[r]["tokens"], feed[r]["root"], None, feed[r]["parents"])
        accept = np.array([got[c][0] for c in range(C)], np.int32)
        assert np.array_equal(as_numpy(node), accept)
        lens, _ = R.kv_commit(host[:2], host[2:], pg.slots, pg.table, lens, accept, feed[r]["parents"])
        assert np.array_equal(as_numpy(new), lens)
        for a, b in zip(after, host):
            assert np.array_equal(as_numpy(a)[0], b)
        moved += sum(len(R.path_of(feed[r]["parents"][c], a)) for c, a in enumerate(accept) if a >= 0)
    assert moved > C
    pg.host = pg.pull()
    n = max(int(lens[s]) for s in pg.slots)
    assert _read(pg, np.zeros(C), nodes=np.array([lens[s] for s in pg.slots], np.int32), sh=sh._replace(n_nodes=n)) == 0
