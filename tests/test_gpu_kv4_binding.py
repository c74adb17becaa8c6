"""The binding of the calls over a 4-bit cache and of the logits' rules on the GPU: every tensor of another type, shape, layout or
device is refused by its name before anything is enqueued, and calls of two streams at once and of two captured graphs
agree with the same calls alone."""

import pytest
import torch

import gated_deltanet_speculative_amd as gdn
from kv4_util import Paged4
from round_util import dev, random_parents

pytestmark = pytest.mark.gpu
BF, FP, I32 = torch.bfloat16, torch.float32, torch.int32
C, N, HQ, HKV, D, LAYERS = 2, 3, 4, 2, 64, 2
zeros = lambda *shape, dtype=I32: torch.zeros(shape, dtype=dtype, device="cuda")  # noqa: E731


def _calls():
    """Per call: the function, its shape and its arguments by name."""
    pg = Paged4(C, N, HQ, HKV, D, 16, BF, [20, 33], layers=LAYERS, seed=1)
    sh, one = pg.sh, gdn.Kv4Cache(*(t[0].contiguous() for t in pg.cache))
    places = dict(slot_ids=dev(pg.slots), page_table=dev(pg.table), seq_len=dev(pg.len))
    tree = dict(parents=zeros(C, N) - 1, lane_nodes=zeros(C) + N)
    q, k = pg.normal(C, N, HQ, D), pg.normal(C, N, HKV, D)
    rope = dict(q=q, k=k, v=k.clone(), inv_freq=zeros(D // 2, dtype=torch.float64), cache=one, **places, positions=zeros(C, N, 2),
                pair_axis=zeros(D // 2), **tree, q_norm=zeros(D, dtype=FP), k_norm=zeros(D, dtype=FP), q_out=torch.empty_like(q),
                status=zeros(1))
    attn = dict(q=q, cache=one, **places, **tree, gate=q.clone(), out=torch.empty_like(q),
                workspace=zeros(gdn.paged_attention_kv4_workspace_size(sh) // 4 + 1, dtype=FP), status=zeros(1))
    commit = dict(caches=pg.cache, **places, accept_node=zeros(C), status=zeros(1), **tree, new_len=zeros(sh.n_slots))
    rows = lambda: zeros(LAYERS, C, N, HKV, D, dtype=BF)  # noqa: E731
    read = dict(caches=pg.cache, slot_ids=places["slot_ids"], page_table=places["page_table"], first_row=zeros(C),
                lane_nodes=tree["lane_nodes"], k_out=rows(), v_out=rows(), status=zeros(1))
    V, P, H, B = 77, 3, 10, 4
    ls = gdn.LogitsShape(C, N, P, V, H, B, BF, FP)
    logits = dict(logits=zeros(C, N, V, dtype=BF), slot_ids=zeros(C), history=zeros(P, H), history_len=zeros(P), prompt_len=zeros(P),
                  repetition=zeros(P, dtype=FP) + 1, presence=zeros(P, dtype=FP), frequency=zeros(P, dtype=FP), bias_tokens=zeros(P, B),
                  bias=zeros(P, B, dtype=FP), temperature=zeros(P, dtype=FP) + 1, mask=zeros(C, N, 3), tokens=zeros(C, N), **tree,
                  out=zeros(C, N, V, dtype=FP), workspace=zeros(gdn.adjust_logits_workspace_size(ls) // 4, dtype=FP), status=zeros(1))
    return {"rope": (gdn.rope_kv4_write, sh, rope), "attn": (gdn.paged_attention_kv4, sh, attn),
            "commit": (gdn.kv4_commit_layers, sh, commit), "read": (gdn.kv4_read_layers, sh, read),
            "logits": (gdn.adjust_logits, ls, logits)}


NEEDED = {"rope": ("q", "k", "v", "inv_freq", "cache", "slot_ids", "page_table", "seq_len"),
          "attn": ("q", "cache", "slot_ids", "page_table", "seq_len"),
          "commit": ("caches", "slot_ids", "page_table", "seq_len", "accept_node", "status"),
          "read": ("caches", "slot_ids", "page_table", "first_row"), "logits": ("logits", "slot_ids")}


@pytest.mark.parametrize("call", ["rope", "attn", "commit", "read", "logits"])
def test_unsuitable_tensors_are_refused(call):
    f, sh, kw = _calls()[call]
    before = {n: t.clone() for n, t in kw.items() if isinstance(t, torch.Tensor)}
    refused = lambda **other: _refused(f, sh, {**kw, **other})  # noqa: E731
    for name, t in kw.items():
        if name in ("cache", "caches"):
            for j in range(4):
                bad = lambda x: type(t)(*(x(y) if i == j else y for i, y in enumerate(t)))  # noqa: E731
                for x in (lambda y: y[..., :-1], lambda y: y.to(I32), lambda y: y.cpu(), lambda y: None, lambda y: y.transpose(-2, -3)):
                    refused(**{name: bad(x)})
            for other in (t.k, t[:3], 5) + (([], [t] * 2, [gdn.Kv4Cache(*(y[0] for y in t))] * 65) if name == "caches" else ()):
                refused(**{name: other})
            continue
        wrong = [t.to(torch.int16), t.cpu(), "text"]
        if name != "workspace":  # (of any shape, and as large as it likes)
            wrong += [t[..., :0], t.unsqueeze(0), torch.cat([t, t[:1]])]
        if t.dim() > 1:
            wrong.append(t.transpose(0, -1))
        else:
            wrong.append(torch.stack([t, t], -1)[..., 0] if t.numel() > 1 else t.expand(2))
        if name in NEEDED[call]:
            wrong.append(None)
        for w in wrong:
            refused(**{name: w})
    torch.cuda.synchronize()
    for n, t in before.items():
        assert torch.equal(kw[n].nan_to_num(), t.nan_to_num()) or n in ("q_out", "out"), f"{n} was written by a refused call"
    f(sh, **kw)  # the call itself is sound
    torch.cuda.synchronize()
    assert int(kw["status"].item()) == 0


def _refused(f, sh, kw):
    with pytest.raises((TypeError, ValueError, gdn.GdnError)):
        f(sh, **kw)


def _pair(seed):
    """An attention call of 17..64 query rows and one of few, over caches of their own, with room for their parts."""
    out = []
    for k, (n, d) in enumerate(((16, 128), (1, 64))):
        pg = Paged4(3, n, 8, 2, d, 16, BF, [700, 350, 1], seed=seed + k)
        parents = random_parents(pg.rng, 3, n)
        args = (pg.normal(3, n, 8, d), pg.cache, dev(pg.slots), dev(pg.table), dev(pg.len))
        out.append((pg, args, dev(parents), gdn.paged_attention_kv4_workspace_size(pg.sh) // 4))
    return out


def test_two_streams_at_once():
    calls = _pair(5)
    alone = [gdn.paged_attention_kv4(pg.sh, *a, parents=p)[0] for pg, a, p, _ in calls]
    outs = [[torch.empty_like(x) for _ in range(8)] for x in alone]
    work = [torch.empty(max(n, 1), dtype=FP, device="cuda") for *_, n in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    for k in range(8):
        for (pg, a, p, _), s, o, w in zip(calls, streams, outs, work):
            with torch.cuda.stream(s):
                gdn.paged_attention_kv4(pg.sh, *a, parents=p, out=o[k], workspace=w)
    torch.cuda.synchronize()
    for x, o in zip(alone, outs):
        assert all(torch.equal(x, y) for y in o)


def test_two_captured_graphs_share_a_workspace():
    """On one stream the graphs follow each other, so what one leaves in the workspace is nothing to the other."""
    calls = _pair(9)
    alone = [gdn.paged_attention_kv4(pg.sh, *a, parents=p)[0] for pg, a, p, _ in calls]
    outs = [torch.empty_like(x) for x in alone]
    work, status = torch.empty(max(1, *(n for *_, n in calls)), dtype=FP, device="cuda"), zeros(1)
    graphs = []
    for (pg, a, p, _), o in zip(calls, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gdn.paged_attention_kv4(pg.sh, *a, parents=p, out=o, workspace=work, status=status)
        graphs.append(g)
    for k in range(4):
        for o in outs:
            o.fill_(-7)
        work.fill_(float("nan"))
        for g in graphs[::-1] if k % 2 else graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, o) for x, o in zip(alone, outs)) and int(status.item()) == 0
