"""Penalties, biases, masks and temperatures on the logits of a draft's nodes against the fp64 oracle: types, sizes of the
vocabulary from one token, draft trees, ragged and padded lanes, tokens and biases that occur twice, ids outside the
vocabulary, rows that a mask leaves empty, infinities and NaN; and the acceptance on the result."""

import numpy as np
import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from gpu_util import log
from oracle import logits_oracle as L
from oracle import round_oracle as R
from round_util import HALF_STEP, SENTINEL, as_numpy, dev, random_parents

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NAMES = ("history", "history_len", "prompt_len", "repetition", "presence", "frequency", "bias_tokens", "bias", "temperature")


class Call:
    """Random inputs of a call with every rule; tests change or drop some."""

    def __init__(self, C, N, V, dtype=BF, out=FP, history=40, bias=5, mask=True, tokens=True, tree=True, temp=True, seed=0, std=3.0,
                 extra=3):
        rng = np.random.default_rng(seed)
        self.rng, P = rng, C + extra
        self.sh = gdn.LogitsShape(C, N, P, V, history, bias, dtype, out)
        self.logits = dev((std * rng.standard_normal((C, N, V))).astype(np.float32), dtype)
        self.slots = rng.permutation(P)[:C].astype(np.int32)
        words = rng.integers(0, V, 12)
        self.rules = dict(P=P)
        if history:
            ids = np.where(rng.random((P, history)) < 0.7, words[rng.integers(0, 12, (P, history))], rng.integers(0, V, (P, history)))
            n = rng.integers(0, history + 1, P)
            self.rules |= dict(history=ids.astype(np.int32), history_len=n.astype(np.int32),
                               prompt_len=(n * rng.random(P)).astype(np.int32))
        self.rules |= dict(repetition=(0.7 + rng.random(P)).astype(np.float32), presence=rng.uniform(-1, 1, P).astype(np.float32),
                           frequency=rng.uniform(-0.5, 0.5, P).astype(np.float32))
        if bias:
            self.rules |= dict(bias_tokens=rng.integers(0, V, (P, bias)).astype(np.int32),
                               bias=rng.uniform(-4, 4, (P, bias)).astype(np.float32))
        if temp:
            self.rules |= dict(temperature=rng.uniform(0.3, 2, P).astype(np.float32))
        self.mask = rng.integers(-2 ** 31, 2 ** 31, (C, N, (V + 31) // 32)).astype(np.int32) if mask else None
        self.tokens = np.where(rng.random((C, N)) < 0.6, words[rng.integers(0, 12, (C, N))], rng.integers(0, V, (C, N))).astype(np.int32) \
            if tokens else None
        self.parents = random_parents(rng, C, N) if tree else None
        self.nodes = None

    def run(self, logits=None, out=None, **kw):
        sh = self.sh
        out = torch.full((sh.n_seqs, sh.n_nodes, sh.vocab), SENTINEL, dtype=sh.out_dtype, device="cuda") if out is None else out
        ws = torch.full((max(1, gdn.adjust_logits_workspace_size(sh) // 4),), float("nan"), device="cuda")
        opt = lambda a: None if a is None else dev(a)  # noqa: E731
        _, status = gdn.adjust_logits(sh, self.logits if logits is None else logits, dev(self.slots),
                                      **{n: opt(self.rules.get(n)) for n in NAMES}, mask=opt(self.mask), tokens=opt(self.tokens),
                                      parents=opt(self.parents), lane_nodes=opt(self.nodes), out=out, workspace=ws, **kw)
        torch.cuda.synchronize()
        return out, int(status.item())

    def want(self, rows=None):
        return L.adjust_logits(as_numpy(self.logits), self.slots, self.rules, self.sh.max_history, self.mask, self.tokens, self.parents,
                               self.nodes, rows)

    def check(self, out=None, status=None, rows=None, expect=0):
        if out is None:
            out, status = self.run()
        res, bits = self.want(rows)
        assert status == bits == expect
        sh, got, worst = self.sh, out, 0.0
        for c in range(sh.n_seqs):
            for i in range(sh.n_nodes):
                if rows is not None and (c, i) not in rows:
                    continue
                g = as_numpy(got[c, i]).astype(np.float64)
                if (c, i) not in res:
                    assert (g == SENTINEL).all(), f"row {(c, i)} was written"
                    continue
                want, tol = expected(*res[c, i], sh)
                assert np.array_equal(np.isnan(g), np.isnan(want)) and np.array_equal(np.isinf(g), np.isinf(want)), (c, i)
                assert np.array_equal(g[np.isinf(g)], want[np.isinf(want)]), (c, i)
                fine = np.isfinite(want)
                if fine.any():
                    ratio = np.abs(g[fine] - want[fine]) / tol[fine]
                    worst = max(worst, float(ratio.max()))
                    assert worst <= 1, f"row {(c, i)} is {worst:.2f} tolerances off at {int(np.argmax(ratio))}"
        return worst


def expected(z, size, T, sh):
    """The row and the largest error of each value.

    z: a sum of at most max_bias + 1 terms, a product with a rounded reciprocal, a fused step and a difference: at most
    max_bias + 6 roundings of a number no larger than `size`.  A probability's exponent (z - max) / T is off by
    twice the largest such error over T and by 2^-22 of itself (the difference's, the factor's and the
    product's rounding), its exponential by 2^-22; the sum of V terms by the same in the mean and by 2^-23 for
    each of at most 80 additions in a row.  One rounding to the type at the end; float16 below 2^-14 has steps of
    2^-24, and exponentials below 2^-126 may be flushed."""
    half = HALF_STEP[sh.out_dtype]
    off = (sh.max_bias + 6) * 2.0 ** -24 * size
    if T is None:
        return z, off + half * np.abs(z) * (1 + 2.0 ** -6) + (2.0 ** -25 if sh.out_dtype is HF else 0) + 1e-35
    want = L.probabilities(z, T)
    if T == 0 or np.isnan(want).any() or not want.any():
        return want, np.full(len(z), 1e-35)
    fine = np.isfinite(z)
    if not fine.any() or np.isposinf(z).any():
        return want, np.full(len(z), 2.0 ** -20)
    e = np.where(fine, (z - z[fine].max()) / T, 0.0)
    arg = 2 * off[fine].max() / T + 2.0 ** -22 * np.abs(e)
    rel = arg + (want * arg).sum() + 2.0 ** -22 + 80 * 2.0 ** -23
    return want, want * rel * (1 + 2.0 ** -6) + half * want * (1 + 2.0 ** -6) + (2.0 ** -25 if sh.out_dtype is HF else 0) + 1e-35


@pytest.mark.parametrize("dtype,out", [(BF, BF), (BF, FP), (HF, HF), (HF, FP), (FP, FP)])
@pytest.mark.parametrize("temp", [False, True])
@pytest.mark.parametrize("V", [1, 7, 33, 1000, 4097, 20011])
def test_types_and_vocabularies(dtype, out, temp, V):
    worst = Call(2, 5, V, dtype, out, temp=temp, seed=V).check()
    log(f"[logits] V={V} {dtype} -> {out} temp={temp}: worst error {worst:.3f} of the tolerance")


@pytest.mark.parametrize("C,N,tree", [(1, 1, False), (3, 32, True), (2, 32, False), (70, 2, True), (1, 9, True)])
@pytest.mark.parametrize("temp", [False, True])
def test_lanes_nodes_and_trees(C, N, tree, temp):
    call = Call(C, N, 2500, tree=tree, temp=temp, seed=C + N, history=300)
    call.check()
    call.nodes = call.rng.integers(0, N + 1, C).astype(np.int32)
    call.check()


@pytest.mark.parametrize("drop", [("history", "history_len", "prompt_len"), ("prompt_len",), ("repetition",), ("presence",), ("frequency",),
                                  ("bias_tokens", "bias"), ("temperature",), ("mask",), ("tokens",), ("parents",), NAMES])
def test_each_rule_is_optional(drop):
    call = Call(2, 6, 999, seed=1)
    for name in drop:
        call.rules.pop(name, None)
        if hasattr(call, name):
            setattr(call, name, None)
    call.check()


def test_each_rule_alone_is_exact_where_it_can_be():
    """Powers of two and small whole numbers: no rounding, so bit for bit."""
    call = Call(1, 3, 500, FP, FP, history=60, bias=0, mask=False, temp=False, seed=2)
    call.logits = dev(call.rng.integers(-8, 9, (1, 3, 500)).astype(np.float32))
    s = call.slots[0]
    call.rules["repetition"][s], call.rules["presence"][s], call.rules["frequency"][s] = 2.0, 0.5, 0.25
    out, status = call.run()
    (res, _) = call.want()
    for i in range(3):
        assert np.array_equal(as_numpy(out[0, i]).astype(np.float64), res[0, i][0])
    # by hand: a token twice in the history behind the prompt and once in it, and on the path of one node
    call.rules["history"][s, :3], call.rules["history_len"][s], call.rules["prompt_len"][s] = 7, 3, 1
    call.tokens, call.parents = np.array([[7, 9, 7]], np.int32), np.array([[-1, -1, 1]], np.int32)
    call.logits[:] = 4.0
    got = as_numpy(call.run()[0])
    assert got[0, 0, 7] == 4 / 2 - 0.25 * 3 - 0.5 and got[0, 1, 7] == 4 / 2 - 0.25 * 2 - 0.5 and got[0, 2, 7] == 4 / 2 - 0.25 * 3 - 0.5
    assert got[0, 0, 9] == 4 and got[0, 1, 9] == got[0, 2, 9] == 4 / 2 - 0.25 - 0.5 and got[0, 0, 8] == 4


@pytest.mark.parametrize("history", [1, 3, 4, 5, 1023, 20000])
def test_histories(history):
    """Long and short, with ids outside the vocabulary, and one token throughout."""
    call = Call(2, 2, 3001, history=history, seed=history)
    h = call.rules["history"]
    h[:, ::3] = call.rng.choice([-1, 3001, 2 ** 31 - 1, -2 ** 31, 3000, 0], h[:, ::3].shape)
    call.rules["history_len"][:] = history
    call.rules["prompt_len"] = call.rng.integers(0, history + 1, call.sh.n_slots).astype(np.int32)
    call.check()
    h[:] = 2999
    call.check()


def test_tokens_and_biases_that_occur_twice():
    call = Call(2, 12, 700, bias=60, seed=5, temp=False)
    call.tokens[:] = call.rng.integers(0, 3, call.tokens.shape)
    call.rules["bias_tokens"][:] = call.rng.choice([5, 6, 699, -1, 700, 2 ** 31 - 1], call.rules["bias_tokens"].shape)
    first, _ = call.run()
    call.check(first, 0)
    for _ in range(3):  # sums in the list's order: the same bits every time
        assert torch.equal(call.run()[0].view(torch.int32), first.view(torch.int32))
    call.rules["bias_tokens"][:] = 5
    call.check()


@pytest.mark.parametrize("dtype,out", [(BF, FP), (FP, FP), (HF, HF)])
def test_rows_that_a_mask_leaves_empty(dtype, out):
    call = Call(2, 4, 333, dtype, out, seed=6)
    call.mask[0, 1], call.mask[1, 3] = 0, 0
    call.mask[0, 2] = 0
    call.mask[0, 2, 10] = 1 << 12  # one token left: the last of the vocabulary
    got, status = call.run()
    call.check(got, status)
    got = as_numpy(got)
    assert (got[0, 1] == 0).all() and (got[1, 3] == 0).all() and got[0, 2, 332] == 1 and got[0, 2, :332].sum() == 0
    call.rules.pop("temperature")
    got = as_numpy(call.run()[0])
    assert np.isneginf(got[0, 1]).all() and np.isneginf(got[0, 2, :332]).all() and np.isfinite(got[0, 2, 332])
    assert call.check() <= 1


@pytest.mark.parametrize("dtype,out", [(BF, FP), (FP, FP), (HF, HF)])
@pytest.mark.parametrize("temp", [None, 1.0, 0.0])
def test_infinities_and_nan(dtype, out, temp):
    """In allowed and in masked places, as logits and as biases."""
    call = Call(1, 8, 600, dtype, out, seed=7, temp=False, bias=3)
    s = call.slots[0]
    call.mask[:] = -1
    call.rules["repetition"][s], call.rules["bias_tokens"][s], call.rules["bias"][s] = 1.5, [50, 51, 52], [-np.inf, 1, 2]
    x = call.logits
    x[0, 0, 100] = x[0, 0, 200] = float("inf")
    x[0, 1, :] = -float("inf")
    x[0, 2, 77] = float("nan")
    x[0, 3, 33], x[0, 3, 34] = float("nan"), float("inf")
    call.mask[0, 3, 1] = ~(3 << 1)  # 33 and 34 are not allowed
    x[0, 4, 5] = -float("inf")
    x[0, 5, :] = float("nan")
    call.mask[0, 5] = 0
    x[0, 6, :] = torch.finfo(dtype).min  # the lowest value of the type is not minus infinity
    call.mask[0, 7] = 0
    x[0, 7, :] = float("inf")
    if temp is not None:
        call.rules["temperature"] = np.full(call.sh.n_slots, temp, np.float32)
    got, status = call.run()
    res, _ = call.want()
    assert status == 0
    g = as_numpy(got).astype(np.float64)
    for i in range(8):
        z, size, T = res[0, i]
        want = z if T is None else L.probabilities(z, T)
        assert np.array_equal(np.isnan(g[0, i]), np.isnan(want)), i
        if i in (1, 5, 7) or T == 0:
            assert np.array_equal(g[0, i], want, equal_nan=True), i
    if temp == 1.0:
        assert g[0, 0, 100] == g[0, 0, 200] == 0.5 and g[0, 0].sum() == 1
        assert np.isnan(g[0, 2]).all() and np.isfinite(g[0, 3]).all() and abs(g[0, 3].sum() - 1) < 2e-3
        assert abs(g[0, 6].sum() - 1) < 2e-3
    if temp == 0.0:
        assert np.isfinite(g).all() and g[0, 0, 100] == 1
    if temp is None:
        assert np.isposinf(g[0, 0, [100, 200]]).all() and np.isnan(g[0, 2, 77]) and np.isneginf(g[0, 3, 33:35]).all()
        assert np.isneginf(g[0, :, 50]).all()


def test_temperature_zero_takes_the_lowest_of_equal_ones():
    call = Call(2, 6, 9001, FP, FP, history=0, bias=0, mask=False, tokens=False, seed=8)
    call.rules = dict(P=call.sh.n_slots, temperature=np.zeros(call.sh.n_slots, np.float32))
    call.logits = dev(call.rng.integers(-4, 5, (2, 6, 9001)).astype(np.float32))  # many equal ones, in every stretch
    got = as_numpy(call.run()[0])
    x = as_numpy(call.logits)
    assert (got.sum(-1) == 1).all() and np.array_equal(got.argmax(-1), x.argmax(-1))
    call.rules["temperature"][call.slots[0]] = 0.7  # lanes of both kinds in one call
    call.check()


@pytest.mark.parametrize("temp", [1e-30, 1e-45, 3e38, 100.0])
def test_temperatures_at_the_ends(temp):
    call = Call(1, 2, 700, FP, FP, seed=9)
    call.rules["temperature"][:] = temp
    got, status = call.run()
    g = as_numpy(got)
    assert status == 0 and np.isfinite(g).all() and np.abs(g.sum(-1) - 1).max() < 1e-5
    call.check(got, status)


def test_padding_invalid_lanes_and_bits():
    C, N = 12, 4
    call = Call(C, N, 300, history=30, seed=10, extra=1)
    call.nodes = np.full(C, N, np.int32)
    r, slots = call.rules, call.slots.copy()
    call.slots[0], call.slots[1], call.nodes[2], call.parents[3, 2] = -1, call.sh.n_slots, N + 1, 2
    call.tokens[4, 1], r["history_len"][slots[5]], r["prompt_len"][slots[6]] = 300, 31, r["history_len"][slots[6]] + 1
    r["repetition"][slots[7]], r["temperature"][slots[8]], r["frequency"][slots[9]] = 0.0, -0.5, np.inf
    res, bits = call.want()
    assert bits == R.SLOT_RANGE | R.NODES | R.PARENT | R.TOKEN | R.LENGTH | L.RULE and {c for c, _ in res} == {10, 11}
    call.check(expect=bits)
    r["presence"][slots[10]] = np.nan
    call.check(expect=bits)
    call.slots[1:] = -1
    call.check()


def test_the_largest_temperature_tells_far_logits_apart():
    call = Call(2, 3, 300, FP, FP, bias=0, history=0, tokens=False, seed=15)
    call.logits *= 2.0 ** 124
    call.rules["temperature"][:] = 3.4e38
    call.check()


@pytest.mark.parametrize("rep", [2.0 ** -126, 2.0 ** -127, 1e-45, 2.0 ** 126, 1.5 * 2.0 ** 126, 2.0 ** 127])
def test_repetitions_at_the_ends(rep):
    """A factor whose reciprocal is no normal number is refused; at the ends of the others no finite result is lost (logits
    of 2^-20 .. 2^-10, so that a quotient by 2^-126 is finite, one by 2^126 loses at most 2^-150)."""
    call = Call(2, 3, 200, FP, FP, bias=0, temp=False, seed=14, mask=False)
    call.logits = call.logits.sign() * 2.0 ** call.logits.abs().clamp(0, 10).neg().sub(10)
    for name in ("presence", "frequency"):
        call.rules[name][:] = 0
    call.rules["repetition"][:] = rep
    call.check(expect=0 if 2.0 ** -126 <= rep <= 2.0 ** 126 else L.RULE)


def test_rows_of_a_padded_vocabulary_and_shared_slots():
    call = Call(3, 4, 501, seed=11)
    wide = torch.full((3, 4, 520), 1e9, dtype=BF, device="cuda")
    wide[:, :, 3:504] = call.logits
    call.check(*call.run(logits=wide[:, :, 3:504]))
    call.slots[:] = call.slots[1]
    call.check()
    with pytest.raises(ValueError, match="evenly strided"):
        gdn.adjust_logits(call.sh, wide[:, :, 3:504].transpose(0, 1).contiguous().transpose(0, 1), dev(call.slots))


def test_guards_around_the_result():
    """An odd vocabulary, out a slice of a larger buffer: nothing in front of it or behind it is written."""
    for out, temp in ((BF, False), (FP, True), (HF, True)):
        call = Call(2, 3, 1237, out, out, seed=12, temp=temp)
        n = 2 * 3 * 1237
        base = torch.full((n + 2001,), SENTINEL, dtype=out, device="cuda")
        call.check(*call.run(out=base[1001:1001 + n].view(2, 3, 1237)))
        assert (as_numpy(base[:1001]) == SENTINEL).all() and (as_numpy(base[1001 + n:]) == SENTINEL).all()


def test_offsets_past_32_bits():
    C, N, V = 70, 32, 1000003  # 2^31 values and more
    call = Call(1, 1, 64, seed=13)
    call.sh = gdn.LogitsShape(C, N, C, V, 0, 0, BF, BF)
    call.logits = torch.randn((C, N, V), device="cuda", dtype=BF, generator=torch.Generator(device="cuda").manual_seed(1))
    call.slots, call.mask, call.parents = np.arange(C, dtype=np.int32), None, None
    call.tokens = call.rng.integers(0, V, (C, N)).astype(np.int32)
    call.rules = dict(P=C, repetition=np.full(C, 1.5, np.float32), temperature=np.full(C, 0.5, np.float32))
    out, status = call.run()
    assert status == 0
    for c, i in ((0, 0), (69, 31), (68, 5), (35, 31)):
        small = call.logits[c:c + 1, i:i + 1].contiguous()
        res, _ = L.adjust_logits(as_numpy(small), [c], call.rules, 0)
        z, size, T = res[0, 0]
        for j in range(i + 1):
            t = call.tokens[c, j]
            z[t] = as_numpy(small)[0, 0, t] * (1.5 if as_numpy(small)[0, 0, t] <= 0 else 1 / 1.5)
        want, tol = expected(z, size * 1.5, T, call.sh)
        # a sum of 10^6 terms: 245 waves' sums of 4096 instead of the 80 additions
        assert (np.abs(as_numpy(out[c, i]) - want) <= tol + want * 400 * 2.0 ** -23).all(), (c, i)


def test_graph_replay_and_another_stream():
    call = Call(3, 8, 5003, seed=14, history=200)
    opt = {n: dev(call.rules[n]) for n in NAMES}
    mask, tokens, parents, slots = dev(call.mask), dev(call.tokens), dev(call.parents), dev(call.slots)
    out, status = torch.zeros(3, 8, 5003, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.adjust_logits_workspace_size(call.sh) // 4, device="cuda")
    x = call.logits.clone()
    run = lambda: gdn.adjust_logits(call.sh, x, slots, **opt, mask=mask, tokens=tokens, parents=parents, out=out, workspace=ws, status=status)  # noqa: E731
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for k in range(4):
        call.logits = dev((3 * call.rng.standard_normal((3, 8, 5003))).astype(np.float32), BF)
        call.tokens = call.rng.integers(0, 5003, (3, 8)).astype(np.int32)
        n = call.rng.integers(0, 201, call.sh.n_slots).astype(np.int32)
        call.rules["history_len"], call.rules["prompt_len"] = n, n // 2
        x.copy_(call.logits)
        tokens.copy_(dev(call.tokens))
        opt["history_len"].copy_(dev(n))
        opt["prompt_len"].copy_(dev(n // 2))
        out.zero_()
        ws.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = call.run()[0]
        assert torch.equal(out, want), f"replay {k}"
    call.check(out, int(status.item()))


@pytest.mark.parametrize("greedy", [False, True])
def test_acceptance_on_the_result(greedy):
    """The rules on the nodes' rows and on the prefix's, and the acceptance of the draft on what they give: the lanes
    accept and draw what the oracle does on the same numbers, and never a token that the grammar forbids."""
    C, N, V = 6, 10, 2003
    call = Call(C, N, V, BF, FP, history=100, seed=15, temp=not greedy, extra=0)
    root = Call(C, 1, V, BF, FP, history=100, seed=16, tree=False, tokens=False, temp=not greedy, extra=0)
    root.rules, root.slots = call.rules, call.slots
    best = lambda row, allowed: int(np.argmax(np.where(allowed, row, -np.inf)))  # noqa: E731
    bits = lambda m: (m.view(np.uint32)[..., np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1  # noqa: E731
    x, x0 = as_numpy(call.logits), as_numpy(root.logits)
    for c in range(C):
        for i in range(N):
            p = call.parents[c, i]
            if call.rng.random() < 0.8:
                call.tokens[c, i] = best(*((x[c, p], bits(call.mask[c, p])) if p >= 0 else (x0[c, 0], bits(root.mask[c, 0]))))
    target, status = call.run()
    call.check(target, status)
    first, status = root.run()
    root.check(first, status)
    u, un = (None, None) if greedy else (dev((0.05 * call.rng.random((C, N))).astype(np.float32)), dev(call.rng.random(C).astype(np.float32)))
    ash = gdn.AcceptShape(C, N, V, FP)
    node, count, token, st = gdn.draft_accept(ash, target, dev(call.tokens), root_target=first[:, 0], parents=dev(call.parents),
                                              slot_ids=dev(call.slots), u_accept=u, u_next=un)
    got, _ = R.draft_accept(as_numpy(target), call.tokens, as_numpy(first[:, 0]), None, call.parents, u_accept=None if greedy else as_numpy(u),
                            u_next=None if greedy else as_numpy(un))
    assert int(st.item()) == 0
    for c in range(C):
        assert (int(node[c]), int(count[c]), int(token[c])) == got[c]
        allowed = bits(call.mask[c, got[c][0]] if got[c][0] >= 0 else root.mask[c, 0])
        assert allowed[got[c][2]]
    assert int(count.sum()) > 0
