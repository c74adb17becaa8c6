"""Cases and plain forms of a round over a key/value cache held in 4 bits, and of the rules applied to its logits.

An attention layer whose paged cache holds keys and values as 4-bit floating point numbers (e2m1) with one power of two
for every 32 values of a row, and what stands between the target's logits and the acceptance of the draft.  A case
names one of these:

  attn    attention of N new tokens per lane (a chain, a draft tree, a prompt chunk) over the 4-bit cache
  rope    rotary positions and the write of the round's keys and values into the 4-bit cache
  commit  the accepted path's rows moved together, in every layer, and the new lengths
  read    rows of the cache of every layer as values
  logits  penalties for repeated tokens, biases and grammar masks on the logits after every node of the draft;
          with temperatures, the probabilities that the acceptance takes

`own = False` computes the plain forms with elementary torch operations in 32 bits (64 for angles); `own = True` makes
the calls of the package.  What the 4-bit cache holds is returned as values, which bfloat16 holds exactly.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # magnitudes of a code's lower three bits; the fourth is the sign
BLOCK = 32


def listed():
    return [
        # one lane of plain decode after a short prompt: the latency of a single call
        dict(name="attn decode 1x1k", op="attn", C=1, N=1, Hq=16, Hkv=2, D=128, ctx=1003, page=16, dtype="bf16",
             tree=False, ragged=False, gate=False),
        # the headline verify round's attention layer: 4 lanes, 16-node trees, a conversation of 8k tokens
        dict(name="attn tree 4x16 8k", op="attn", C=4, N=16, Hq=32, Hkv=8, D=128, ctx=8192, page=64, dtype="bf16",
             tree=True, ragged=False, gate=False),
        # a full server's decode step: 64 lanes with long caches of different lengths, what a small cache is for
        dict(name="attn decode 64x32k", op="attn", C=64, N=1, Hq=32, Hkv=4, D=128, ctx=32768, page=64, dtype="f16",
             tree=False, ragged=True, gate=False),
        # two prompts' next chunks behind long caches, wide heads, closing sigmoid gate
        dict(name="attn chunk 2x2048 16k", op="attn", C=2, N=2048, Hq=16, Hkv=2, D=256, ctx=16384, page=128,
             dtype="bf16", tree=False, ragged=True, gate=True),
        # the decode step's rotation and cache write for 4 lanes
        dict(name="rope decode 4", op="rope", C=4, N=1, Hq=32, Hkv=8, D=128, rot=128, axes=1, norm=False, ctx=5000,
             page=64, xdtype="bf16", dtype="bf16", tree=False, interleaved=False),
        # a prompt with images: three axes, part of a wide head rotated, q and k normed, 32-bit activations
        dict(name="rope prompt 2x4096", op="rope", C=2, N=4096, Hq=16, Hkv=2, D=256, rot=64, axes=3, norm=True,
             ctx=100, page=128, xdtype="f32", dtype="bf16", tree=False, interleaved=False),
        # the headline round's commit over 16 attention layers
        dict(name="commit 4x16 l16", op="commit", C=4, N=16, Hkv=8, D=128, layers=16, ctx=500, page=64, dtype="bf16",
             tree=True),
        # the commit of a full server's 32-node trees
        dict(name="commit 64x32 l16", op="commit", C=64, N=32, Hkv=8, D=128, layers=16, ctx=150, page=64, dtype="bf16",
             tree=True),
        # the round's rows of one layer looked at
        dict(name="read 4x16 l1", op="read", C=4, N=16, Hkv=8, D=128, layers=1, ctx=5000, page=64, dtype="bf16"),
        # a sequence of 4095 tokens leaves the 4-bit cache for one of 16 bits, every layer
        dict(name="read 1x4095 l16", op="read", C=1, N=4095, Hkv=8, D=128, layers=16, ctx=0, page=48, dtype="f16"),
        # plain greedy decode of 4 lanes: penalties over a conversation, some biases; the logits themselves
        dict(name="logits decode 4", op="logits", C=4, N=1, V=32768, history=2000, bias=20, mask=False, tokens=False,
             tree=False, temp=False, ragged=False, dtype="bf16", out="bf16"),
        # the headline round's trees under a grammar, a large odd vocabulary, probabilities for the acceptance
        dict(name="logits tree 4x16", op="logits", C=4, N=16, V=130001, history=8192, bias=300, mask=True, tokens=True,
             tree=True, temp=True, ragged=False, dtype="bf16", out="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn"] * 4 + ["logits"] * 3 + ["rope", "commit", "read"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    page = rng.choice([16, 32, 48, 64, 100, 128, 256])
    if op == "attn":
        kind = rng.choice(["decode", "tree", "chain", "chunk"])
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8])
        C = _log(rng, 1, 64) if kind != "chunk" else _log(rng, 1, 4)
        N = {"decode": 1, "tree": rng.randint(2, 32), "chain": rng.randint(2, 32), "chunk": _log(rng, 33, 4096)}[kind]
        case = dict(op=op, C=C, N=N, Hq=Hq, Hkv=Hkv, D=D, ctx=_log(rng, 1, 32768), page=page, dtype=dtype,
                    tree=kind == "tree", ragged=rng.random() < 0.6, gate=rng.random() < 0.3)
        while (work(case)["flops"] > (1e11 if dtype == "f32" else 4e11) or C * Hkv * D * (case["ctx"] + N) > 1.1e9
               or C * Hq * N * (case["ctx"] + N) > 1.2e9):
            if case["ctx"] > N:
                case["ctx"] //= 2
            else:
                case["N"] = N = max(1, N // 2)
        return case
    if op == "logits":
        kind = rng.choice(["decode", "tree", "chain"])
        N = 1 if kind == "decode" else rng.randint(2, 32)
        C, V = _log(rng, 1, 64), _log(rng, 1000, 200000)
        while C * N * V > 4e7:
            C, N = max(1, C // 2), N if C > 1 else max(1, N // 2)
        return dict(op=op, C=C, N=N, V=V, history=_log(rng, 1, 32768), bias=rng.choice([0, rng.randint(1, 300)]),
                    mask=rng.random() < 0.5, tokens=kind != "decode" or rng.random() < 0.3, tree=kind == "tree" and N > 1,
                    temp=rng.random() < 0.6, ragged=rng.random() < 0.4, dtype=dtype, out=rng.choice([dtype, "f32"]))
    if op == "rope":
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        tree = rng.random() < 0.4
        return dict(op=op, C=_log(rng, 1, 16), N=rng.randint(1, 32) if tree else _log(rng, 1, 1024),
                    Hq=Hkv * rng.choice([1, 2, 3, 8]), Hkv=Hkv, D=D, rot=16 * rng.randint(1, D // 16),
                    axes=rng.choice([1, 1, 2, 3]), norm=rng.random() < 0.5, ctx=_log(rng, 1, 4000), page=page,
                    xdtype=rng.choice([dtype, "f32"]), dtype=dtype, tree=tree, interleaved=rng.random() < 0.3)
    case = dict(op=op, C=_log(rng, 1, 64 if op == "commit" else 8), N=rng.randint(1, 32) if op == "commit" else _log(rng, 1, 4000),
                Hkv=rng.choice([1, 2, 4, 8]), D=rng.choice([64, 128, 256]), layers=rng.randint(1, 24), ctx=_log(rng, 1, 300),
                page=page, dtype=dtype)
    if op == "commit":
        case["tree"] = rng.random() < 0.8
    values = case["C"] * (case["N"] + (case["ctx"] + page if op == "commit" else page)) * case["Hkv"] * case["D"]
    case["layers"] = max(1, min(case["layers"], int(1.2e8 / values)))
    return case


def _lens(case):
    """Committed tokens of each lane: all `ctx`, or spread between ctx / 2 and ctx."""
    C, ctx = case["C"], case["ctx"]
    return [ctx - (c * ctx) // (2 * C) if case.get("ragged") else ctx for c in range(C)]


def _counts(case):
    """Present tokens of each lane: ragged lanes have from N down to N / 2 of them."""
    C, N = case["C"], case["N"]
    return [N - (c * N) // (2 * C) if case.get("ragged") else N for c in range(C)]


def work(case):
    C, N, es = case["C"], case["N"], SIZE[case["dtype"]]
    if case["op"] == "logits":
        vals = sum(_counts(case)) * case["V"]
        return {"bytes": vals * (es + SIZE[case["out"]] + (0.125 if case["mask"] else 0)) + 4 * C * (case["history"] + 2 * case["bias"]),
                "flops": (8.0 if case["temp"] else 4.0) * vals}
    D, Hkv = case["D"], case["Hkv"]
    row = D // 2 + D // BLOCK  # bytes of a row's codes and scales
    if case["op"] == "attn":
        Hq = case["Hq"]
        lens, counts = _lens(case), _counts(case)
        # a tree's node sees about log2(N) + 1 ancestors, a chain's half the chain
        seen = lambda n: n * (math.log2(n) + 1) if case["tree"] else n * (n + 1) / 2  # noqa: E731
        pairs = sum(n * length + seen(n) for n, length in zip(counts, lens))
        rows = sum(n + length for n, length in zip(counts, lens))
        return {"bytes": 2 * Hkv * rows * row + (2 + bool(case["gate"])) * Hq * sum(counts) * D * es, "flops": 4.0 * D * Hq * pairs}
    # the other three give the rows they wrote, moved or read as values of 16 or 32 bits
    if case["op"] == "rope":
        vals = C * N * D * (case["Hq"] + 2 * Hkv)
        return {"bytes": vals * SIZE[case["xdtype"]] + C * N * (Hkv * 2 * (row + 2 * D) + case["Hq"] * D * es) + 4 * C * N * case["axes"],
                "flops": C * N * ((case["Hq"] + Hkv) * (3.0 * case["rot"] + (3.0 * D if case["norm"] else 0)) + 2 * Hkv * 2.0 * D)}
    rows = 2 * case["layers"] * C * N * Hkv
    if case["op"] == "read":
        return {"bytes": rows * (row + es * D), "flops": 1.0 * rows * D}
    # a random tree's path has about log2(N) / 2 + 1 rows that move
    moved = 2 * case["layers"] * C * (math.log2(N) / 2 + 1) * case["tree"] * Hkv
    return {"bytes": 2 * moved * row + rows * (row + 2 * D) + 12 * C * N + 8 * C, "flops": 0}


# ---------------------------------------------------------------- inputs
def _random_parents(rs, C, N):
    """Draft trees: node i hangs on the committed prefix (-1) or on any earlier node."""
    u = rs.random_sample((C, N))
    return (np.floor(u * (np.arange(N) + 1)) - 1).astype(np.int32)


def _paged(case, rs, lens, extra):
    """Slots, page table and lengths: every lane's pages scattered over the pool, unused entries -1."""
    C, page = case["C"], case["page"]
    P = C + 3
    need = [-(-(n + extra) // page) for n in lens]
    n_pages, max_pages = sum(need) + 5, max(need)
    slots = rs.permutation(P)[:C].astype(np.int32)
    ids = rs.permutation(n_pages)
    table, length = np.full((P, max_pages), -1, np.int32), np.zeros(P, np.int32)
    at = 0
    for c in range(C):
        table[slots[c], :need[c]] = ids[at:at + need[c]]
        length[slots[c]] = lens[c]
        at += need[c]
    return P, n_pages, max_pages, slots, table, length


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _random_cache(gen, layers, n_pages, Hkv, page, D):
    """Codes and scales of normally distributed rows, made in pieces."""
    codes = torch.empty(layers * n_pages, Hkv, page, D // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(layers * n_pages, Hkv, page, D // BLOCK, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    for at in range(0, layers * n_pages, step):
        x = torch.randn((len(codes[at:at + step]), Hkv, page, D), generator=gen, device="cuda")
        codes[at:at + step], scales[at:at + step] = _quantised(x, 125)
    return codes.view(layers, n_pages, Hkv, page, D // 2), scales.view(layers, n_pages, Hkv, page, D // BLOCK)


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=dt, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)

    C, N = case["C"], case["N"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "parents": None, "lane_nodes": None}
    if case.get("tree"):
        s["parents"] = _gpu(_random_parents(rs, C, N))
    if case.get("ragged"):
        s["lane_nodes"] = _gpu(np.array(_counts(case), np.int32))
    if case["op"] == "logits":
        return _prepare_logits(case, s, rs, gen)
    lens = [int(v) for v in rs.permutation(_lens(case))]
    P, n_pages, max_pages, slots, table, length = _paged(case, rs, lens, N)
    s |= {"slots": _gpu(slots), "table": _gpu(table), "len": _gpu(length), "longest": max(lens)}
    Hkv, D, page, layers = case["Hkv"], case["D"], case["page"], case.get("layers", 1)
    s["dims"] = (C, N, P, case.get("Hq", Hkv), Hkv, D, page, n_pages, max_pages, dt)
    s["grid"] = torch.tensor(GRID + tuple(-v for v in GRID), device="cuda")
    s["k"], s["ks"] = _random_cache(gen, layers, n_pages, Hkv, page, D)
    s["v"], s["vs"] = _random_cache(gen, layers, n_pages, Hkv, page, D)
    s["layer"] = [s[n][0] for n in ("k", "ks", "v", "vs")]
    # the rows that a user looks at afterwards: behind the committed ones, or from the front
    s["first"] = _gpu(np.array([length[p] if case["op"] != "read" else 0 for p in slots], np.int32))
    if case["op"] != "attn":
        value = dt if case["op"] == "read" else torch.bfloat16
        s["rows_k"], s["rows_v"] = (torch.zeros(layers, C, N, Hkv, D, dtype=value, device="cuda") for _ in range(2))
    if case["op"] == "read":
        return s
    if case["op"] == "commit":
        s["accept"] = _gpu(rs.randint(max(-1, N // 2 - 1), N, C).astype(np.int32))
        s["new_len"] = torch.zeros(P, dtype=torch.int32, device="cuda")
        return s
    Hq = case["Hq"]
    if case["op"] == "attn":
        s["q"] = randn(C, N, Hq, D, std=2.0)  # scores of a few units, as after a norm of q and k
        s["out"] = torch.zeros(C, N, Hq, D, dtype=dt, device="cuda")
        s["gate"] = randn(C, N, Hq, D) if case["gate"] else None
        s["work"] = torch.empty(1 << 26, dtype=torch.float32, device="cuda")  # the program's scratch, 256 MiB
        return s
    x = randn(C, N, Hq + 2 * Hkv, D, dtype=DTYPES[case["xdtype"]])  # the stacked q | k | v projection
    s["q"], s["kx"], s["vx"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    s["q_out"] = torch.zeros(C, N, Hq, D, dtype=dt, device="cuda")
    half = case["rot"] // 2
    s["inv_freq"] = _gpu(1e6 ** (-np.arange(half) / half))
    s["axis"] = s["positions"] = None
    if case["axes"] > 1:  # positions of text and image patches deep in a long session
        s["axis"] = _gpu((np.arange(half) % case["axes"]).astype(np.int32))
        base = rs.randint(0, 1 << 20, (C, 1, 1))
        s["positions"] = _gpu((base + rs.randint(0, 2000, (C, N, case["axes"]))).astype(np.int32))
    s["q_norm"], s["k_norm"] = (1 + randn(D, dtype=torch.float32, std=0.1) if case["norm"] else None for _ in range(2))
    return s


def _prepare_logits(case, s, rs, gen):
    C, N, V, H = case["C"], case["N"], case["V"], case["history"]
    P = C + 3
    slots = rs.permutation(P)[:C].astype(np.int32)
    # a conversation repeats its tokens: most of them are drawn from a few hundred
    words = rs.randint(0, V, 400)
    history = np.where(rs.random_sample((P, H)) < 0.8, words[rs.randint(0, 400, (P, H))], rs.randint(0, V, (P, H)))
    length = np.array([H - (p * H) // (3 * P) for p in range(P)])
    s |= {"slots": _gpu(slots), "history": _gpu(history.astype(np.int32)), "hist_len": _gpu(length.astype(np.int32)),
          "prompt_len": _gpu((length * rs.random_sample(P)).astype(np.int32))}
    s["logits"] = torch.randn((C, N, V), generator=gen, device="cuda").mul_(3.0).to(DTYPES[case["dtype"]])
    s["repetition"] = _gpu((1 + 0.3 * rs.random_sample(P)).astype(np.float32))
    s["presence"], s["frequency"] = (_gpu((0.8 * rs.random_sample(P)).astype(np.float32)) for _ in range(2))
    s["bias_tokens"] = s["bias"] = s["mask"] = s["tokens"] = s["temperature"] = s["work"] = None
    if case["bias"]:
        some = np.stack([rs.permutation(V)[:case["bias"]] for _ in range(P)])
        s["bias_tokens"], s["bias"] = _gpu(some.astype(np.int32)), _gpu(rs.uniform(-8, 4, some.shape).astype(np.float32))
    if case["mask"]:  # a grammar allows a half or a quarter of the tokens
        words = torch.randint(-(1 << 31), 1 << 31, (2, C, N, (V + 31) // 32), generator=gen, device="cuda")
        s["mask"] = (words[0] & torch.where(words[1, :, :, :1] > 0, words[1], -1)).int()
    if case["tokens"]:  # drafted tokens, some of them of the conversation
        near = history[slots[:, None], rs.randint(0, H, (C, N))]
        s["tokens"] = _gpu(np.where(rs.random_sample((C, N)) < 0.5, near, rs.randint(0, V, (C, N))).astype(np.int32))
    if case["temp"]:  # most lanes sample, every fifth is greedy
        s["temperature"] = _gpu(np.where(np.arange(P) % 5 == 4, 0.0, rs.uniform(0.3, 1.5, P)).astype(np.float32))
    s["out"] = torch.zeros(C, N, V, dtype=DTYPES[case["out"]], device="cuda")
    s["work"] = torch.empty(1 << 22, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"attn": _attn, "rope": _rope, "commit": _commit, "read": _read, "logits": _logits}[s["case"]["op"]](s)


def _own(s):
    import gated_deltanet_speculative_amd as gdn

    case, op = s["case"], s["case"]["op"]
    if op == "logits":
        sh = gdn.LogitsShape(case["C"], case["N"], case["C"] + 3, case["V"], case["history"], case["bias"],
                             DTYPES[case["dtype"]], DTYPES[case["out"]])
        out, _ = gdn.adjust_logits(sh, s["logits"], s["slots"], history=s["history"], history_len=s["hist_len"],
                                   prompt_len=s["prompt_len"], repetition=s["repetition"], presence=s["presence"],
                                   frequency=s["frequency"], bias_tokens=s["bias_tokens"], bias=s["bias"], mask=s["mask"],
                                   tokens=s["tokens"], parents=s["parents"], lane_nodes=s["lane_nodes"],
                                   temperature=s["temperature"], out=s["out"], workspace=s["work"], status=s["status"])
        return {"out": out}
    sh = gdn.AttnShape(*s["dims"])
    layer, caches = gdn.Kv4Cache(*s["layer"]), gdn.Kv4Cache(s["k"], s["ks"], s["v"], s["vs"])
    if op == "attn":
        out, _ = gdn.paged_attention_kv4(sh, s["q"], layer, s["slots"], s["table"], s["len"], parents=s["parents"],
                                         lane_nodes=s["lane_nodes"], gate=s["gate"], gate_mode=1, out=s["out"],
                                         workspace=s["work"], status=s["status"])
        return {"out": out}
    got = {}
    if op == "rope":
        got["q"], _ = gdn.rope_kv4_write(sh, s["q"], s["kx"], s["vx"], s["inv_freq"], layer, s["slots"], s["table"],
                                         s["len"], positions=s["positions"], pair_axis=s["axis"], parents=s["parents"],
                                         lane_nodes=s["lane_nodes"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6,
                                         interleaved=case["interleaved"], q_out=s["q_out"], status=s["status"])
    if op == "commit":
        got["len"] = gdn.kv4_commit_layers(sh, caches, s["slots"], s["table"], s["len"], s["accept"], s["status"],
                                           parents=s["parents"], lane_nodes=s["lane_nodes"], new_len=s["new_len"])
    got["k"], got["v"], _ = gdn.kv4_read_layers(sh._replace(dtype=s["rows_k"].dtype), caches, s["slots"], s["table"], s["first"],
                                                k_out=s["rows_k"], v_out=s["rows_v"], status=s["status"])
    return got


# ---------------------------------------------------------------- plain forms
def _quantised(x, most):
    """Codes and scales of rows whose last axis is made of blocks: the block's power of two is that of its largest
    magnitude rounded to one fraction bit, two below; ties of a code go to the even one."""
    y = x.float().unflatten(-1, (-1, BLOCK))
    m, e = torch.frexp(y.abs().amax(-1))
    e = (torch.where(m == 0, -200, e - 3 + (m >= 0.875).int())).clamp(-125, most)
    y = torch.ldexp(y, -e[..., None])
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).byte()
    code = (code + 8 * (y < 0).byte()).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, (e + 127).byte()


def _values(s, codes, scales):
    """What codes and scales stand for, in 32 bits."""
    x = s["grid"][torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    return (x.unflatten(-1, (-1, BLOCK)) * torch.exp2(scales.float() - 127.0)[..., None]).flatten(-2)


def _ancestors(parents, C, N, device):
    """[C, N, N] truth values: j is i or an ancestor of i.  The sum of the powers of the parent matrix."""
    if parents is None:
        return torch.ones(N, N, dtype=torch.bool, device=device).tril().expand(C, N, N)
    one = torch.eye(N, device=device)
    up = (parents[:, :, None] == torch.arange(N, device=device)).float()
    up2 = up @ up
    up4 = up2 @ up2
    up8 = up4 @ up4
    return ((one + up) @ (one + up2) @ (one + up4) @ (one + up8) @ (one + up8 @ up8)) > 0


def _places(s, pos):
    """Page and place in the page of the cache rows `pos` [C, T] of each lane."""
    page = s["case"]["page"]
    table = s["table"][s["slots"].long()].long()
    return table.gather(1, pos // page).clamp(min=0), pos % page


def _attn(s):
    C, N, _, Hq, Hkv, D, page, _, max_pages, dt = s["dims"]
    dev, G, T = s["q"].device, Hq // Hkv, s["longest"] + N
    length = s["len"][s["slots"].long()].long()
    pos = torch.arange(T, device=dev).expand(C, T)
    pages, at = _places(s, pos)
    k = _values(s, s["k"][0][pages, :, at], s["ks"][0][pages, :, at]).permute(0, 2, 3, 1).contiguous()  # [C, Hkv, D, T]
    q = s["q"].float().view(C, N, Hkv, G, D).transpose(1, 2).reshape(C, Hkv, N * G, D)
    x = (q @ k).mul_(D ** -0.5)
    del k
    count = torch.full((C,), N, device=dev) if s["lane_nodes"] is None else s["lane_nodes"].long()
    node = pos - length[:, None]  # the round's node at this row, if any
    inside = (node >= 0) & (node < count[:, None])
    tree = _ancestors(s["parents"], C, N, dev)
    seen = tree.gather(2, node.clamp(0, N - 1)[:, None, :].expand(C, N, T)) & inside[:, None, :] | (node < 0)[:, None, :]
    seen = seen.view(C, 1, N, 1, T)
    x = x.view(C, Hkv, N, G, T).masked_fill_(~seen, -torch.inf)
    x = x.sub_(x.amax(-1, keepdim=True)).exp_()
    x = x.div_(x.sum(-1, keepdim=True)).view(C, Hkv, N * G, T)
    v = _values(s, s["v"][0][pages, :, at], s["vs"][0][pages, :, at]).transpose(1, 2).contiguous()  # [C, Hkv, T, D]
    o = (x @ v).view(C, Hkv, N, G, D).transpose(1, 2).reshape(C, N, Hq, D)
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    present = torch.arange(N, device=dev)[None, :] < count[:, None]
    return {"out": torch.where(present[:, :, None, None], o, 0.0).to(dt)}


def _read(s):
    """The rows behind `first`, of every layer."""
    C, N = s["case"]["C"], s["case"]["N"]
    pages, at = _places(s, s["first"].long()[:, None] + torch.arange(N, device=s["first"].device))
    return {n: _values(s, s[n][:, pages, :, at], s[n + "s"][:, pages, :, at]).permute(2, 0, 1, 3, 4).to(s["rows_k"].dtype)
            for n in ("k", "v")}


def _rms(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w


def _rotate(x, cos, sin, rot, interleaved):
    half = rot // 2
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :half], x[..., half:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned, x[..., rot:]), -1)


def _rope(s):
    C, N, _, Hq, Hkv, D, page, _, _, dt = s["dims"]
    case, dev = s["case"], s["q"].device
    length = s["len"][s["slots"].long()].long()
    i = torch.arange(N, device=dev)
    if s["positions"] is None:
        depth = _ancestors(s["parents"], C, N, dev).sum(-1) - 1 if s["parents"] is not None else i.expand(C, N)
        p = (length[:, None] + depth)[:, :, None].expand(C, N, case["rot"] // 2)
    else:
        p = s["positions"][:, :, s["axis"].long()]
    angle = p.double() * s["inv_freq"]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    q = _rotate(_rms(s["q"], s["q_norm"]), cos, sin, case["rot"], case["interleaved"])
    k = _rotate(_rms(s["kx"], s["k_norm"]), cos, sin, case["rot"], case["interleaved"])
    pages, at = _places(s, length[:, None] + i)
    most = 13 if dt == torch.float16 else 125
    s["k"][0][pages, :, at], s["ks"][0][pages, :, at] = _quantised(k, most)
    s["v"][0][pages, :, at], s["vs"][0][pages, :, at] = _quantised(s["vx"], most)
    return {"q": q.to(dt), **_read(s)}


def _commit(s):
    C, N, P, _, Hkv, D, page, _, _, dt = s["dims"]
    dev, accept, slots = s["k"].device, s["accept"].long(), s["slots"].long()
    i = torch.arange(N, device=dev)
    tree = _ancestors(s["parents"], C, N, dev)
    path = tree[torch.arange(C, device=dev), accept.clamp(min=0)] & (accept >= 0)[:, None]  # [C, N]
    length = s["len"][slots].long()[:, None]
    src = _places(s, length + i)
    dst = _places(s, length + torch.where(path, path.cumsum(-1) - 1, i))
    (sp, so), (dp, do) = ((a[path], b[path]) for a, b in (src, dst))
    s["k"][:, dp, :, do], s["ks"][:, dp, :, do] = s["k"][:, sp, :, so], s["ks"][:, sp, :, so]
    s["v"][:, dp, :, do], s["vs"][:, dp, :, do] = s["v"][:, sp, :, so], s["vs"][:, sp, :, so]
    s["new_len"].copy_(s["len"]).index_add_(0, slots, path.sum(-1).int())
    return {"len": s["new_len"], **_read(s)}


def _logits(s):
    case = s["case"]
    C, N, V = case["C"], case["N"], case["V"]
    dev, slots = s["logits"].device, s["slots"].long()
    past = s["history"][slots].long()
    at = torch.arange(past.shape[1], device=dev)
    there = at < s["hist_len"][slots][:, None]
    made = there & (at >= s["prompt_len"][slots][:, None])
    seen, count = (torch.zeros(C, V, device=dev).scatter_add_(1, past, t.float())[:, None] for t in (there, made))
    if s["tokens"] is not None:  # the tokens on a node's path have been generated for it
        path = _ancestors(s["parents"], C, N, dev).float()
        on_path = torch.zeros(C, N, V, device=dev).scatter_add_(2, s["tokens"].long()[:, None, :].expand(C, N, N), path)
        seen, count = seen + on_path, count + on_path
    x = s["logits"].float()
    if s["bias"] is not None:
        x = x + torch.zeros(C, V, device=dev).scatter_add_(1, s["bias_tokens"][slots].long(), s["bias"][slots])[:, None]
    r, f, p = (s[n][slots][:, None, None] for n in ("repetition", "frequency", "presence"))
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - f * count - p * (count > 0)
    if s["mask"] is not None:
        v = torch.arange(V, device=dev)
        x = torch.where((s["mask"][:, :, v // 32] >> (v % 32)) & 1 > 0, x, -torch.inf)
    if s["temperature"] is not None:
        t = s["temperature"][slots][:, None, None]
        top = x.amax(-1, keepdim=True)
        y = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
        y = y / y.sum(-1, keepdim=True)
        v = torch.arange(V, device=dev)
        x = torch.where(t > 0, y, (v == torch.where(x == top, v, V).amin(-1, keepdim=True)).float())
    if s["lane_nodes"] is not None:
        x = torch.where((torch.arange(N, device=dev) < s["lane_nodes"][:, None])[:, :, None], x, 0.0)
    return {"out": x.to(s["out"].dtype)}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "commit": _exact_commit, "read": _exact_read,
            "logits": _exact_logits}[case["op"]](case, s)


def _host(t):
    return None if t is None else t.cpu().numpy()


def _path(parents, i):
    """The nodes from the prefix's child down to node i; without parents a chain."""
    if parents is None:
        return list(range(i + 1))
    got = []
    while i >= 0:
        got.append(i)
        i = int(parents[i])
    return got[::-1]


def _lane_rows(case, s, c, n):
    """Page and place of lane c's first n cached tokens."""
    t = torch.arange(n, device="cuda")
    return s["table"][int(s["slots"][c])].long()[t // case["page"]], t % case["page"]


def _exact_values(codes, scales):
    """From the numbers' bits: sign, two exponent bits with bias 1 (0: no leading one), one fraction bit."""
    def half(n):
        n = n.long()
        e, f = n >> 1 & 3, (n & 1).double()
        mag = torch.where(e > 0, (1 + f / 2) * torch.pow(2.0, (e - 1).double()), f / 2)
        return torch.where(n & 8 > 0, -mag, mag)

    out = torch.zeros(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    out[..., 0::2], out[..., 1::2] = half(codes & 15), half(codes // 16)
    return out * torch.pow(2.0, scales.double() - 127).repeat_interleave(BLOCK, -1)


def _nearest(x, most):
    """The value of the 4-bit form of every x."""
    b = x.reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    a = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0)))
    e = torch.where(a >= torch.pow(2.0, e + 1), e + 1, torch.where(a < torch.pow(2.0, e), e - 1, e))
    e = torch.where(a / torch.pow(2.0, e) >= 1.75, e + 1, e) - 2
    e = torch.where(a > 0, e, -125.0).clamp(-125, most)
    y = b / torch.pow(2.0, e)
    # the grid's step at this magnitude, and the nearest multiple of it (torch rounds halves to even)
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    return ((torch.round(y / step) * step).clamp(-6, 6) * torch.pow(2.0, e)).reshape(x.shape)


def _exact_attn(case, s):
    C, N, G, D = case["C"], case["N"], case["Hq"] // case["Hkv"], case["D"]
    parents, counts = _host(s["parents"]), _host(s["lane_nodes"])
    out = torch.zeros(C, N, case["Hq"], D, dtype=torch.float64, device="cuda")
    for c in range(C):
        n, length = N if counts is None else int(counts[c]), int(s["len"][s["slots"][c].long()])
        allowed = torch.zeros(n, length + n, dtype=torch.bool, device="cuda")
        if parents is None:
            allowed = torch.ones(n, length + n, dtype=torch.bool, device="cuda").tril(length)
        else:
            allowed[:, :length] = True
            for i in range(n):
                allowed[i, [length + j for j in _path(parents[c], i)]] = True
        rows = _lane_rows(case, s, c, length + n)
        for h in range(case["Hkv"]):
            k, v = (_exact_values(s[name][0][rows[0], h, rows[1]], s[name + "s"][0][rows[0], h, rows[1]]) for name in "kv")
            for g in range(G):
                x = s["q"][c, :n, h * G + g].double() @ k.T.contiguous() / math.sqrt(D)
                x = torch.softmax(torch.where(allowed, x, -math.inf), -1)
                out[c, :n, h * G + g] = x @ v
    return {"out": out if s["gate"] is None else out / (1 + torch.exp(-s["gate"].double()))}


def _exact_rows(case, s, k, v):
    """Rows first .. first + N - 1 of every lane, from [layers][pages][heads][page][...] pairs of codes and scales."""
    got = {}
    for name, (codes, scales) in (("k", k), ("v", v)):
        lanes = []
        for c in range(case["C"]):
            first = int(s["first"][c])
            pages, at = (t[first:] for t in _lane_rows(case, s, c, first + case["N"]))
            lanes.append(torch.stack([_exact_values(codes[l][pages, :, at], scales[l][pages, :, at]) for l in range(len(codes))]))
        got[name] = torch.stack(lanes, 1)
    return got


def _exact_read(case, s):
    return _exact_rows(case, s, (s["k"], s["ks"]), (s["v"], s["vs"]))


def _exact_rope(case, s):
    C, N, half = case["C"], case["N"], case["rot"] // 2
    parents = _host(s["parents"])
    pos = torch.zeros(C, N, half, dtype=torch.float64, device="cuda")
    for c in range(C):
        length = int(s["len"][s["slots"][c].long()])
        if s["positions"] is None:
            depth = np.arange(N) if parents is None else [len(_path(parents[c], i)) - 1 for i in range(N)]
            pos[c] = torch.tensor([length + int(v) for v in depth], dtype=torch.float64, device="cuda")[:, None]
        else:
            for j in range(half):
                pos[c, :, j] = s["positions"][c, :, int(j % case["axes"])].double()
    turn = torch.polar(torch.ones_like(pos), pos * s["inv_freq"])[:, :, None]

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.double()
        at = (torch.arange(half, device="cuda") * 2, torch.arange(half, device="cuda") * 2 + 1)
        if not case["interleaved"]:
            at = (torch.arange(half, device="cuda"), torch.arange(half, device="cuda") + half)
        z = torch.complex(x[..., at[0]], x[..., at[1]]) * turn
        y = x.clone()
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        return y

    most = 13 if case["dtype"] == "f16" else 125
    return {"q": one(s["q"], s["q_norm"]), "k": _nearest(one(s["kx"], s["k_norm"]), most)[None],
            "v": _nearest(s["vx"].double(), most)[None]}


def _exact_commit(case, s):
    parents, accept = _host(s["parents"]), _host(s["accept"])
    moved, new_len = {n: s[n].clone() for n in ("k", "ks", "v", "vs")}, s["len"].clone()
    for c in range(case["C"]):
        slot = int(s["slots"][c])
        length, path = int(s["len"][slot]), _path(None if parents is None else parents[c], int(accept[c]))
        pages, at = _lane_rows(case, s, c, length + case["N"])
        for j, i in enumerate(path):
            for n, t in moved.items():
                t[:, pages[length + j], :, at[length + j]] = s[n][:, pages[length + i], :, at[length + i]]
        new_len[slot] = length + len(path)
    return {"len": new_len, **_exact_rows(case, s, (moved["k"], moved["ks"]), (moved["v"], moved["vs"]))}


def _exact_logits(case, s):
    C, N, V = case["C"], case["N"], case["V"]
    h = {n: _host(s[n]) for n in ("parents", "lane_nodes", "slots", "history", "hist_len", "prompt_len", "repetition", "presence",
                                  "frequency", "bias_tokens", "bias", "mask", "tokens", "temperature")}
    out = torch.zeros(C, N, V, dtype=torch.float64)
    for c in range(C):
        p = h["slots"][c]
        n, prompt = int(h["hist_len"][p]), int(h["prompt_len"][p])
        seen0, made0 = (np.bincount(t, minlength=V) for t in (h["history"][p, :n], h["history"][p, prompt:n]))
        for i in range(N if h["lane_nodes"] is None else int(h["lane_nodes"][c])):
            x = s["logits"][c, i].double().cpu().numpy()
            if h["bias"] is not None:
                x[h["bias_tokens"][p]] += h["bias"][p].astype(np.float64)  # (no token twice)
            seen, made = seen0.copy(), made0.copy()
            if h["tokens"] is not None:
                for j in _path(None if h["parents"] is None else h["parents"][c], i):
                    seen[h["tokens"][c, j]] += 1
                    made[h["tokens"][c, j]] += 1
            r = float(h["repetition"][p])
            some = np.nonzero(seen)[0]
            x[some] = np.where(x[some] > 0, x[some] / r, x[some] * r)
            x -= float(h["frequency"][p]) * made + float(h["presence"][p]) * np.minimum(made, 1)
            if h["mask"] is not None:
                bits = np.unpackbits(h["mask"][c, i].view(np.uint8), bitorder="little")[:V]
                x[bits == 0] = -np.inf
            if h["temperature"] is not None:
                t = float(h["temperature"][p])
                if t > 0:
                    x = np.exp((x - x.max()) / t)
                    x /= x.sum()
                else:
                    one = np.zeros(V)
                    one[int(np.argmax(x))] = 1
                    x = one
            out[c, i] = torch.from_numpy(x)
    return {"out": out}
