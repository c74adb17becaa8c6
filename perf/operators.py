"""Cases and plain forms of the operators that surround the recurrence in a speculative round.

A round of the draft-tree route needs more than the recurrence of its gated delta rule layers: the
model's attention layers write the round's keys and values into a paged cache (rotary positions),
attend over it with the draft tree's mask, the drafted tokens are tested against the target's
probabilities, and the accepted path's cache rows are moved together.  A case names one of these:

  attn    attention of N new tokens per lane (a chain, a draft tree, a prompt chunk) over a paged cache
  rope    rotary positions (one to three axes, optional norm of q and k) and the write into the cache
  accept  drafted tokens against the target's probabilities, with given random numbers (or greedy)
  commit  the accepted path's cache rows moved together, in every layer, and the new lengths

`own = False` computes the plain forms with elementary torch operations in 32 bits (64 for angles,
probabilities and running sums); `own = True` makes the calls of the package.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one lane of plain decode after a short prompt: the latency of a single call
        dict(name="attn decode 1x1k", op="attn", C=1, N=1, Hq=16, Hkv=2, D=128, ctx=1003, page=16, dtype="bf16",
             tree=False, ragged=False, gate=False),
        # the headline verify round's attention layer: 4 lanes, 16-node trees, a conversation of 8k tokens
        dict(name="attn tree 4x16 8k", op="attn", C=4, N=16, Hq=32, Hkv=8, D=128, ctx=8192, page=64, dtype="bf16",
             tree=True, ragged=False, gate=False),
        # a full server's decode step: 64 lanes with long caches of different lengths
        dict(name="attn decode 64x32k", op="attn", C=64, N=1, Hq=32, Hkv=4, D=128, ctx=32768, page=64, dtype="f16",
             tree=False, ragged=True, gate=False),
        # a prompt into an empty cache
        dict(name="attn prompt 1x4096", op="attn", C=1, N=4096, Hq=32, Hkv=8, D=128, ctx=0, page=64, dtype="bf16",
             tree=False, ragged=False, gate=False),
        # two prompts' next chunks behind long caches, wide heads, closing sigmoid gate
        dict(name="attn chunk 2x2048 16k", op="attn", C=2, N=2048, Hq=16, Hkv=2, D=256, ctx=16384, page=128,
             dtype="bf16", tree=False, ragged=True, gate=True),
        # the 5-lane round of 8-token chains in 32 bits, odd lengths, pages that are no power of two
        dict(name="attn chain 5x8 f32", op="attn", C=5, N=8, Hq=8, Hkv=8, D=64, ctx=2999, page=48, dtype="f32",
             tree=False, ragged=True, gate=False),
        # the decode step's rotation and cache write for 4 lanes
        dict(name="rope decode 4", op="rope", C=4, N=1, Hq=32, Hkv=8, D=128, rot=128, axes=1, norm=False, ctx=5000,
             page=64, xdtype="bf16", dtype="bf16", tree=False, interleaved=False),
        # a prompt with images: three axes, part of a wide head rotated, q and k normed, 32-bit activations
        dict(name="rope prompt 2x4096", op="rope", C=2, N=4096, Hq=16, Hkv=2, D=256, rot=64, axes=3, norm=True,
             ctx=100, page=128, xdtype="f32", dtype="bf16", tree=False, interleaved=False),
        # 8 lanes of 8-token chains drawn from the drafter's distribution, a large odd vocabulary
        dict(name="accept chain 8x8", op="accept", C=8, N=8, V=130001, dtype="f32", tree=False, draft=True, root=False,
             greedy=False),
        # the headline round's trees of candidate tokens
        dict(name="accept tree 4x16", op="accept", C=4, N=16, V=32768, dtype="bf16", tree=True, draft=False, root=True,
             greedy=False),
        # the headline round's commit over 16 attention layers
        dict(name="commit 4x16 l16", op="commit", C=4, N=16, Hkv=8, D=128, layers=16, ctx=500, page=64, dtype="bf16",
             tree=True),
        # the commit of a full server's 32-node trees
        dict(name="commit 64x32 l16", op="commit", C=64, N=32, Hkv=8, D=128, layers=16, ctx=150, page=64, dtype="bf16",
             tree=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn"] * 4 + ["rope", "accept", "accept", "commit"])
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
        while (work(case)["flops"] > (1e11 if dtype == "f32" else 4e11) or work(case)["bytes"] > 2e9
               or C * Hq * N * (case["ctx"] + N) > 1.2e9):
            if case["ctx"] > N:
                case["ctx"] //= 2
            else:
                case["N"] = N = max(1, N // 2)
        return case
    if op == "rope":
        D = rng.choice([64, 128, 256])
        Hkv = rng.choice([1, 2, 4, 8])
        tree = rng.random() < 0.4
        return dict(op=op, C=_log(rng, 1, 16), N=rng.randint(1, 32) if tree else _log(rng, 1, 1024),
                    Hq=Hkv * rng.choice([1, 2, 3, 8]), Hkv=Hkv, D=D, rot=16 * rng.randint(1, D // 16),
                    axes=rng.choice([1, 1, 2, 3]), norm=rng.random() < 0.5, ctx=_log(rng, 1, 4000), page=page,
                    xdtype=rng.choice([dtype, "f32"]), dtype=dtype, tree=tree, interleaved=rng.random() < 0.3)
    if op == "accept":
        tree, greedy = rng.random() < 0.5, rng.random() < 0.3
        return dict(op=op, C=_log(rng, 1, 32), N=rng.randint(1, 32 if tree else 12), V=_log(rng, 1000, 200000),
                    dtype=rng.choice(["f32", "f32", "bf16", "f16"]), tree=tree,
                    draft=not tree and not greedy and rng.random() < 0.7, root=rng.random() < 0.5, greedy=greedy)
    case = dict(op=op, C=_log(rng, 1, 64), N=rng.randint(1, 32), Hkv=rng.choice([1, 2, 4, 8]),
                D=rng.choice([64, 128, 256]), layers=rng.randint(1, 24), ctx=_log(rng, 1, 300), page=page,
                dtype=dtype, tree=rng.random() < 0.8)
    rows = case["C"] * (case["ctx"] + case["N"] + page)
    case["layers"] = max(1, min(case["layers"], int(1e9 / (rows * case["Hkv"] * case["D"] * SIZE[dtype]))))
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
    if case["op"] == "attn":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        lens, counts = _lens(case), _counts(case)
        # a tree's node sees about log2(N) + 1 ancestors, a chain's half the chain
        seen = lambda n: n * (math.log2(n) + 1) if case["tree"] else n * (n + 1) / 2  # noqa: E731
        pairs = sum(n * length + seen(n) for n, length in zip(counts, lens))
        rows = sum(n + length for n, length in zip(counts, lens))
        return {"bytes": es * D * (2 * Hkv * rows + (2 + bool(case["gate"])) * Hq * sum(counts)),
                "flops": 4.0 * D * Hq * pairs}
    if case["op"] == "rope":
        vals = C * N * case["D"] * (case["Hq"] + 2 * case["Hkv"])
        return {"bytes": vals * (SIZE[case["xdtype"]] + es) + 4 * C * N * case["axes"],
                "flops": C * N * (case["Hq"] + case["Hkv"]) * (3.0 * case["rot"] + (3.0 * case["D"] if case["norm"] else 0))}
    if case["op"] == "accept":
        rows = C * (N + case["root"]) if case["greedy"] else C * (1 + case["draft"])
        return {"bytes": es * rows * case["V"], "flops": 2.0 * rows * case["V"]}
    # a random tree's path has about log2(N) / 2 + 1 rows that move
    moved = C * (math.log2(N) / 2 + 1) * case["tree"]
    return {"bytes": 2 * 2 * es * case["layers"] * moved * case["Hkv"] * case["D"] + 12 * C * N + 8 * C, "flops": 0}


# ---------------------------------------------------------------- inputs
def _random_parents(rs, C, N, pending):
    """Draft trees: node i hangs on the committed prefix (-1) or on any earlier node; where the first node is a
    pending token, every other one descends from it."""
    i = np.arange(N)
    u = rs.random_sample((C, N))
    return (np.floor(u * i) - (i == 0) if pending else np.floor(u * (i + 1)) - 1).astype(np.int32)


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


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, dtype=dt, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype).mul_(std)

    C, N = case["C"], case["N"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "parents": None, "lane_nodes": None}
    if case["tree"]:
        s["parents"] = _gpu(_random_parents(rs, C, N, case["op"] == "accept" and not case["root"]))
    if case["op"] == "accept":
        return _prepare_accept(case, s, rs, gen)
    if case.get("ragged"):
        s["lane_nodes"] = _gpu(np.array(_counts(case), np.int32))
    lens = [int(v) for v in rs.permutation(_lens(case))]
    P, n_pages, max_pages, slots, table, length = _paged(case, rs, lens, N)
    s |= {"slots": _gpu(slots), "table": _gpu(table), "len": _gpu(length), "longest": max(lens)}
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    s["dims"] = (C, N, P, case.get("Hq", Hkv), Hkv, D, page, n_pages, max_pages, dt)
    if case["op"] == "commit":
        s["k"], s["v"] = (randn(case["layers"], n_pages, Hkv, page, D) for _ in range(2))
        s["accept"] = _gpu(rs.randint(max(-1, N // 2 - 1), N, C).astype(np.int32))
        s["new_len"] = torch.zeros(P, dtype=torch.int32, device="cuda")
        return s
    Hq = case["Hq"]
    s["k_cache"], s["v_cache"] = randn(n_pages, Hkv, page, D), randn(n_pages, Hkv, page, D)
    if case["op"] == "attn":
        s["q"] = randn(C, N, Hq, D, std=2.0)  # scores of a few units, as after a norm of q and k
        s["out"] = torch.zeros(C, N, Hq, D, dtype=dt, device="cuda")
        s["gate"] = randn(C, N, Hq, D) if case["gate"] else None
        s["work"] = torch.empty(1 << 26, dtype=torch.float32, device="cuda")  # the program's scratch, 256 MiB
        return s
    x = randn(C, N, Hq + 2 * Hkv, D, dtype=DTYPES[case["xdtype"]])  # the stacked q | k | v projection
    s["x"] = x
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


def _prepare_accept(case, s, rs, gen):
    C, N, V, dt = case["C"], case["N"], case["V"], DTYPES[case["dtype"]]
    logits = torch.randn((C, N + 1, V), generator=gen, device="cuda").mul_(3.0)  # row 0: the committed prefix
    p = torch.softmax(logits, -1)
    logits.add_(torch.randn((C, N + 1, V), generator=gen, device="cuda"))  # the drafter's guess of the same rows
    q = torch.softmax(logits, -1)
    del logits
    par = s["parents"].long() if case["tree"] else torch.arange(-1, N - 1, device="cuda").expand(C, N)
    rank = (par[:, :, None] == par[:, None, :]).tril(-1).sum(-1)  # how many earlier siblings
    if case["draft"]:
        tokens = torch.multinomial(q[:, :N].reshape(C * N, V), 1, generator=gen).reshape(C, N)
    else:  # candidates: the drafter's most likely tokens, one for each sibling
        top = q.topk(min(33, V), -1).indices
        tokens = top[torch.arange(C, device="cuda")[:, None], par + 1, rank]
    s["tokens"] = tokens.int().contiguous()
    s["target"] = p[:, 1:].to(dt).contiguous()
    s["root"] = p[:, 0].to(dt).contiguous() if case["root"] else None
    s["draft"] = q[:, :N].to(dt).contiguous() if case["draft"] else None
    s["u"] = s["u_next"] = None
    if not case["greedy"]:
        s["u"], s["u_next"] = torch.rand((C, N), generator=gen, device="cuda"), torch.rand(C, generator=gen, device="cuda")
    s["out"] = [torch.zeros(C, dtype=torch.int32, device="cuda") for _ in range(3)]
    s["work"] = torch.empty(1 << 21, dtype=torch.float32, device="cuda")
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        return _own(s)
    return {"attn": _attn, "rope": _rope, "accept": _accept, "commit": _commit}[s["case"]["op"]](s)


def _own(s):
    import gated_deltanet_speculative_amd as gdn

    case, op = s["case"], s["case"]["op"]
    if op == "accept":
        sh = gdn.AcceptShape(case["C"], case["N"], case["V"], DTYPES[case["dtype"]])
        accept, count, token, _ = gdn.draft_accept(
            sh, s["target"], s["tokens"], root_target=s["root"], draft=s["draft"], parents=s["parents"], u_accept=s["u"],
            u_next=s["u_next"], accept_node=s["out"][0], n_accept=s["out"][1], next_token=s["out"][2],
            workspace=s["work"], status=s["status"])
        return {"accept": accept, "count": count, "token": token}
    sh = gdn.AttnShape(*s["dims"])
    if op == "attn":
        out, _ = gdn.paged_attention(sh, s["q"], s["k_cache"], s["v_cache"], s["slots"], s["table"], s["len"],
                                     parents=s["parents"], lane_nodes=s["lane_nodes"], gate=s["gate"], gate_mode=1,
                                     out=s["out"], workspace=s["work"], status=s["status"])
        return {"out": out}
    if op == "rope":
        q_out, _ = gdn.rope_kv_write(sh, s["q"], s["kx"], s["vx"], s["inv_freq"], s["k_cache"], s["v_cache"], s["slots"],
                                     s["table"], s["len"], positions=s["positions"], pair_axis=s["axis"],
                                     parents=s["parents"], lane_nodes=s["lane_nodes"], q_norm=s["q_norm"],
                                     k_norm=s["k_norm"], eps=1e-6, interleaved=case["interleaved"], q_out=s["q_out"],
                                     status=s["status"])
        return {"q": q_out, "k": s["k_cache"], "v": s["v_cache"]}
    new_len = gdn.kv_commit_layers(sh, s["k"], s["v"], s["slots"], s["table"], s["len"], s["accept"], s["status"],
                                   parents=s["parents"], lane_nodes=s["lane_nodes"], new_len=s["new_len"])
    return {"k": s["k"], "v": s["v"], "len": new_len}


# ---------------------------------------------------------------- plain forms
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


def _rows(s, pos):
    """Page and place in the page of the cache rows `pos` [C, T] of each lane."""
    page = s["case"]["page"]
    table = s["table"][s["slots"].long()].long()
    return table.gather(1, pos // page).clamp(min=0), pos % page


def _attn(s):
    C, N, _, Hq, Hkv, D, page, _, max_pages, dt = s["dims"]
    dev, G, T = s["q"].device, Hq // Hkv, s["longest"] + N
    length = s["len"][s["slots"].long()].long()
    pos = torch.arange(T, device=dev).expand(C, T)
    pages, at = _rows(s, pos)
    k = s["k_cache"][pages, :, at].float().permute(0, 2, 3, 1).contiguous()  # [C, Hkv, D, T]
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
    v = s["v_cache"][pages, :, at].float().transpose(1, 2).contiguous()  # [C, Hkv, T, D]
    o = (x @ v).view(C, Hkv, N, G, D).transpose(1, 2).reshape(C, N, Hq, D)
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    present = torch.arange(N, device=dev)[None, :] < count[:, None]
    return {"out": torch.where(present[:, :, None, None], o, 0.0).to(dt)}


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
    case, dev = s["case"], s["x"].device
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
    pages, at = _rows(s, length[:, None] + i)
    s["k_cache"][pages, :, at] = k.to(dt)
    s["v_cache"][pages, :, at] = s["vx"].to(dt)
    return {"q": q.to(dt), "k": s["k_cache"], "v": s["v_cache"]}


def _best(x):
    """The lowest index of each row's largest value."""
    x = x.float().nan_to_num(nan=-torch.inf, posinf=torch.inf, neginf=-torch.inf)
    at = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, x.shape[-1]).amin(-1)


def _accept(s):
    case = s["case"]
    C, N, V = case["C"], case["N"], case["V"]
    dev, target, root, x = s["target"].device, s["target"], s["root"], s["tokens"].long()
    c, i = torch.arange(C, device=dev), torch.arange(N, device=dev)
    par = s["parents"].long() if s["parents"] is not None else (i - 1).expand(C, N)
    earlier = (par[:, :, None] == par[:, None, :]) & (i[None, :] < i[:, None])  # [C, i, j]: j is an earlier sibling of i
    again = (earlier & (x[:, :, None] == x[:, None, :])).any(-1)
    if case["greedy"]:
        best = torch.cat((_best(target), _best(root)[:, None] if root is not None else torch.full((C, 1), -1, device=dev)), 1)
        ok = (x == best.gather(1, torch.where(par < 0, N, par))) & ~again
    else:
        p = target[c[:, None], par.clamp(min=0), x].double()
        if root is not None:
            p = torch.where(par < 0, root[c[:, None], x].double(), p)
        p = torch.where((p > 0) & ~again, p, 0.0)
        left = 1.0 - (earlier * p[:, None, :]).sum(-1)
        q = s["draft"][c[:, None], i, x].double() if s["draft"] is not None else 1.0
        ok = s["u"].double() * q * left < p
    if root is None:  # the first node on the prefix is the token already drawn
        ok = torch.where(par < 0, ~earlier.any(-1), ok)
    ok = ok & ~(earlier & ok[:, None, :]).any(-1)
    taken = ~(_ancestors(par, C, N, dev) & ~ok[:, None, :]).any(-1)
    accept = torch.where(taken, i, -1).amax(-1)
    row = target[c, accept.clamp(min=0)]
    if root is not None:
        row = torch.where((accept < 0)[:, None], root, row)
    if case["greedy"]:
        token = _best(row)
    else:
        p = row.double()
        p = torch.where(p > 0, p, 0.0)
        child = par == accept[:, None]
        if s["draft"] is not None:
            last = accept == N - 1  # no child: nothing was refused
            w = (p - s["draft"][c, (accept + 1).clamp(max=N - 1)].double() * ~last[:, None]).clamp(min=0)
        else:
            w = p * (torch.zeros(C, V, device=dev).scatter_add_(1, x, child.float()) == 0)
        w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
        run_sum = w.cumsum(-1)
        at = (run_sum <= s["u_next"].double()[:, None] * run_sum[:, -1:]).sum(-1)
        last_one = torch.where(w > 0, torch.arange(V, device=dev), -1).amax(-1)
        token = torch.minimum(at, last_one)
    return {"accept": accept.int(), "count": taken.sum(-1).int(), "token": token.int()}


def _commit(s):
    C, N, P, _, Hkv, D, page, _, _, dt = s["dims"]
    dev, accept, slots = s["k"].device, s["accept"].long(), s["slots"].long()
    i = torch.arange(N, device=dev)
    tree = _ancestors(s["parents"], C, N, dev)
    path = tree[torch.arange(C, device=dev), accept.clamp(min=0)] & (accept >= 0)[:, None]  # [C, N]
    length = s["len"][slots].long()[:, None]
    src = _rows(s, length + i)
    dst = _rows(s, length + torch.where(path, path.cumsum(-1) - 1, i))
    (sp, so), (dp, do) = ((a[path], b[path]) for a, b in (src, dst))
    s["k"][:, dp, :, do] = s["k"][:, sp, :, so]
    s["v"][:, dp, :, do] = s["v"][:, sp, :, so]
    s["new_len"].copy_(s["len"]).index_add_(0, slots, path.sum(-1).int())
    return {"k": s["k"], "v": s["v"], "len": s["new_len"]}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "rope": _exact_rope, "accept": _exact_accept, "commit": _exact_commit}[case["op"]](case, s)


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
    """Flat row numbers (page * page_size + place) of lane c's first n cached tokens."""
    t = torch.arange(n, device="cuda")
    return s["table"][int(s["slots"][c])].long()[t // case["page"]], t % case["page"]


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
            k, v = (s[name][rows[0], h, rows[1]].double() for name in ("k_cache", "v_cache"))
            for g in range(G):
                x = s["q"][c, :n, h * G + g].double() @ k.T.contiguous() / math.sqrt(D)
                x = torch.softmax(torch.where(allowed, x, -math.inf), -1)
                out[c, :n, h * G + g] = x @ v
    return {"out": out if s["gate"] is None else out / (1 + torch.exp(-s["gate"].double()))}


def _exact_rope(case, s):
    C, N, half = case["C"], case["N"], case["rot"] // 2
    parents = _host(s["parents"])
    pos = torch.zeros(C, N, half, dtype=torch.float64, device="cuda")
    got = {"k": s["k_cache"].double(), "v": s["v_cache"].double()}
    length = [int(s["len"][s["slots"][c].long()]) for c in range(C)]
    for c in range(C):
        if s["positions"] is None:
            depth = np.arange(N) if parents is None else [len(_path(parents[c], i)) - 1 for i in range(N)]
            pos[c] = torch.tensor([length[c] + int(v) for v in depth], dtype=torch.float64, device="cuda")[:, None]
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

    k = one(s["kx"], s["k_norm"])
    for c in range(C):
        pages, at = (t[length[c]:] for t in _lane_rows(case, s, c, length[c] + N))
        got["k"][pages, :, at], got["v"][pages, :, at] = k[c], s["vx"][c].double()
    return {"q": one(s["q"], s["q_norm"]), **got}


def _exact_accept(case, s):
    C, N, V = case["C"], case["N"], case["V"]
    parents, tokens, u, u_next = (_host(s[n]) for n in ("parents", "tokens", "u", "u_next"))
    accepts, counts, nexts = [], [], []
    for c in range(C):
        par = [i - 1 for i in range(N)] if parents is None else [int(v) for v in parents[c]]
        node, count = -1, 0
        while True:
            row = s["target"][c, node] if node >= 0 else s["root"][c] if s["root"] is not None else None
            row = None if row is None else row.double().cpu().numpy()
            kids, went, left, refused = [j for j in range(N) if par[j] == node], None, 1.0, []
            best = None if row is None else int(np.argmax(row))
            for j in kids:
                t = int(tokens[c, j])
                if row is None:
                    went = kids[0]
                elif case["greedy"]:
                    went = j if t == best else None
                elif t not in refused:
                    q = float(s["draft"][c, j, t].double()) if case["draft"] else 1.0
                    if float(u[c, j]) * q * left < row[t]:
                        went = j
                    else:
                        left -= row[t]
                        refused.append(t)
                if went is not None:
                    break
            if went is None:
                break
            node, count = went, count + 1
        if case["greedy"]:
            token = best
        else:
            w = row.copy()
            if case["draft"] and kids:
                w = np.maximum(row - s["draft"][c, kids[0]].double().cpu().numpy(), 0)
            w[refused if not case["draft"] else []] = 0
            w = w if w.sum() > 0 else row
            total = np.cumsum(w)
            token = min(int(np.searchsorted(total, float(u_next[c]) * total[-1], side="right")), int(np.nonzero(w)[0][-1]))
        accepts.append(node), counts.append(count), nexts.append(token)
    return {"accept": torch.tensor(accepts, dtype=torch.int32), "count": torch.tensor(counts, dtype=torch.int32),
            "token": torch.tensor(nexts, dtype=torch.int32)}


def _exact_commit(case, s):
    parents, accept = _host(s["parents"]), _host(s["accept"])
    k, v, new_len = s["k"].double(), s["v"].double(), s["len"].clone()
    for c in range(case["C"]):
        slot = int(s["slots"][c])
        length, path = int(s["len"][slot]), _path(None if parents is None else parents[c], int(accept[c]))
        pages, at = _lane_rows(case, s, c, length + case["N"])
        for j, i in enumerate(path):
            for t, src in ((k, s["k"]), (v, s["v"])):
                t[:, pages[length + j], :, at[length + j]] = src[:, pages[length + i], :, at[length + i]].double()
        new_len[slot] = length + len(path)
    return {"k": k, "v": v, "len": new_len}
