"""Times of the gdn_round.h calls over the cases of perf/operators.py, beside their floors; with --more of the gdn_kv4.h and
gdn_logits.h calls over those of perf/more_operators.py.

    python -m gated_deltanet_speculative_amd.round_times [--more] [--only TEXT] [--further] [--draw N --seed S] [--plain] [--errors]

Prints per case the microseconds of one pass among others (calls through the Python binding one after the other,
over three sets of inputs in turn; the median of five loops) and the floor of these inputs: the larger of bytes / the rate of a large
copy and operations / the rate of a large matrix product of the type, both measured first.  --further adds cases that
the file does not list, --draw N cases drawn from its ranges with the given seed.  --plain also times the plain forms,
--errors gives the distance from the definition in 64 bits (2-norm of the difference over that of the result).

    rocprofv3 --kernel-trace --stats --output-format csv -- python3 -m gated_deltanet_speculative_amd.round_times --passes 18
    python -m gated_deltanet_speculative_amd.round_times --summary KERNEL_TRACE_CSV [FETCH_CSV WRITE_CSV]

The first runs each case without timing it, for a profiler (with --pmc FETCH_SIZE and --pmc WRITE_SIZE for the counters);
the second prints each case's kernels from the CSV files: median duration, read and written MB as the counters report
them.  Both take --more, --only, --further, --draw and --seed, which have to be the same.
"""

from __future__ import annotations

import argparse
import csv
import importlib.util
import os
import random
import re
import statistics

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DTYPES = ("f32", "bf16", "f16")

_WIDE = dict(op="attn", D=256, page=64, dtype="bf16", gate=True)
FURTHER = [
    # the verify route's wide gated heads: plain decode, draft trees
    dict(_WIDE, name="attn decode 4x8k wide", C=4, N=1, Hq=16, Hkv=2, ctx=8192, tree=False, ragged=False),
    dict(_WIDE, name="attn decode 64x8k wide", C=64, N=1, Hq=16, Hkv=2, ctx=8192, tree=False, ragged=True),
    dict(_WIDE, name="attn tree 4x16 8k wide", C=4, N=16, Hq=24, Hkv=4, ctx=8192, tree=True, ragged=False),
    # a page table for 128k rows over a short cache, and the same calls with a table as long as the cache
    dict(name="attn decode 1x1k, table of 128k", op="attn", C=1, N=1, Hq=16, Hkv=2, D=128, ctx=1003, page=16, dtype="bf16",
         tree=False, ragged=False, gate=False, rows=1 << 17),
    dict(name="attn tree 4x16 1k", op="attn", C=4, N=16, Hq=32, Hkv=8, D=128, ctx=1000, page=64, dtype="bf16", tree=True,
         ragged=False, gate=False),
    dict(name="attn tree 4x16 1k, table of 128k", op="attn", C=4, N=16, Hq=32, Hkv=8, D=128, ctx=1000, page=64, dtype="bf16",
         tree=True, ragged=False, gate=False, rows=1 << 17),
    # float32 at the other widths
    dict(name="attn chain 5x8 f32 128", op="attn", C=5, N=8, Hq=8, Hkv=8, D=128, ctx=2999, page=48, dtype="f32", tree=False,
         ragged=True, gate=False),
    dict(name="attn chain 5x8 f32 256", op="attn", C=5, N=8, Hq=8, Hkv=8, D=256, ctx=2999, page=48, dtype="f32", tree=False,
         ragged=True, gate=False),
    # greedy acceptance reads every row of a lane
    dict(name="accept greedy tree 4x16", op="accept", C=4, N=16, V=130001, dtype="bf16", tree=True, draft=False, root=True,
         greedy=True),
    dict(name="accept greedy chain 8x8 f32", op="accept", C=8, N=8, V=32768, dtype="f32", tree=False, draft=False, root=True,
         greedy=True),
    # wide heads' commit
    dict(name="commit 4x16 l16 wide", op="commit", C=4, N=16, Hkv=2, D=256, layers=16, ctx=500, page=64, dtype="bf16", tree=True),
]
# over a 4-bit cache
FURTHER_MORE = [
    dict(_WIDE, name="attn decode 64x8k wide", C=64, N=1, Hq=16, Hkv=2, ctx=8192, tree=False, ragged=True),
    dict(_WIDE, name="attn tree 4x16 8k wide", C=4, N=16, Hq=24, Hkv=4, ctx=8192, tree=True, ragged=False),
    dict(name="attn tree 1x16 8k", op="attn", C=1, N=16, Hq=32, Hkv=8, D=128, ctx=8192, page=64, dtype="bf16", tree=True,
         ragged=False, gate=False),
    dict(name="attn tree 4x16 1k", op="attn", C=4, N=16, Hq=32, Hkv=8, D=128, ctx=1000, page=64, dtype="bf16", tree=True,
         ragged=False, gate=False),
    dict(name="attn chain 5x8 f32 256", op="attn", C=5, N=8, Hq=8, Hkv=8, D=256, ctx=2999, page=48, dtype="f32", tree=False,
         ragged=True, gate=False),
    # a page table for 128k rows over a short cache, and over one of 8192 tokens
    dict(name="attn decode 1x1k, table of 128k", op="attn", C=1, N=1, Hq=16, Hkv=2, D=128, ctx=1003, page=16, dtype="bf16",
         tree=False, ragged=False, gate=False, rows=1 << 17),
    dict(name="attn tree 4x16 1k, table of 128k", op="attn", C=4, N=16, Hq=32, Hkv=8, D=128, ctx=1000, page=64, dtype="bf16",
         tree=True, ragged=False, gate=False, rows=1 << 17),
    dict(name="attn tree 1x16 8k, table of 128k", op="attn", C=1, N=16, Hq=32, Hkv=8, D=128, ctx=8192, page=64, dtype="bf16",
         tree=True, ragged=False, gate=False, rows=1 << 17),
    # more than 16 query rows in float32
    dict(name="attn tree 4x16 8k f32", op="attn", C=4, N=16, Hq=32, Hkv=8, D=128, ctx=8192, page=64, dtype="f32", tree=True,
         ragged=False, gate=False),
    dict(name="attn tree 4x16 8k f32 256", op="attn", C=4, N=16, Hq=24, Hkv=4, D=256, ctx=8192, page=64, dtype="f32", tree=True,
         ragged=False, gate=False),
    dict(name="attn chunk 1x1024 4k f32", op="attn", C=1, N=1024, Hq=16, Hkv=4, D=64, ctx=4096, page=64, dtype="f32", tree=False,
         ragged=False, gate=False),
    # chunks of the narrower heads, and prompts into an empty cache
    dict(name="attn chunk 2x2048 16k, 128", op="attn", C=2, N=2048, Hq=32, Hkv=8, D=128, ctx=16384, page=64, dtype="bf16",
         tree=False, ragged=False, gate=False),
    dict(name="attn chunk 2x2048 16k, 64", op="attn", C=2, N=2048, Hq=32, Hkv=8, D=64, ctx=16384, page=64, dtype="f16", tree=False,
         ragged=False, gate=False),
    dict(name="attn prompt 1x4096", op="attn", C=1, N=4096, Hq=32, Hkv=8, D=128, ctx=0, page=64, dtype="bf16", tree=False,
         ragged=False, gate=False),
    dict(name="attn prompt 1x1417, 64", op="attn", C=1, N=1417, Hq=8, Hkv=8, D=64, ctx=0, page=64, dtype="bf16", tree=False,
         ragged=False, gate=False),
    dict(name="attn prompt 1x1164, 256", op="attn", C=1, N=1164, Hq=9, Hkv=3, D=256, ctx=0, page=64, dtype="bf16", tree=False,
         ragged=False, gate=False),
    # many rows of logits, and vocabularies within one stretch
    dict(name="logits tree 32x32, no temperature", op="logits", C=32, N=32, V=130001, history=8192, bias=300, mask=True, tokens=True,
         tree=True, temp=False, ragged=False, dtype="bf16", out="bf16"),
    dict(name="logits tree 32x32", op="logits", C=32, N=32, V=130001, history=8192, bias=300, mask=True, tokens=True, tree=True,
         temp=True, ragged=False, dtype="bf16", out="f32"),
    dict(name="logits tree 52x32 small", op="logits", C=52, N=32, V=1092, history=2000, bias=20, mask=True, tokens=True, tree=True,
         temp=True, ragged=False, dtype="bf16", out="f32"),
    dict(name="logits chain 1x22 small", op="logits", C=1, N=22, V=1220, history=24000, bias=20, mask=True, tokens=True, tree=False,
         temp=True, ragged=False, dtype="bf16", out="f32"),
]


def operators(more=False):
    """The cases' file, as a module."""
    name = "more_operators.py" if more else "operators.py"
    spec = importlib.util.spec_from_file_location("round_operators", os.path.join(ROOT, "perf", name))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def cases(ops, further=False, draws=0, seed=0, only=""):
    rng = random.Random(seed)
    drawn = [dict(ops.draw(rng), name=f"draw {k}") for k in range(draws)]
    beside = FURTHER if ops.__file__.endswith(os.sep + "operators.py") else FURTHER_MORE
    return [c for c in (*ops.listed(), *(beside if further else ()), *drawn) if only in c["name"]]


def prepare(ops, case, seed):
    """The case's inputs; with `rows`, under a page table for that many."""
    s = ops.prepare(case, seed)
    if "rows" in case:
        entries, d = case["rows"] // case["page"], list(s["dims"])
        s["table"] = torch.nn.functional.pad(s["table"], (0, entries - d[8]), value=-1)
        d[8] = entries
        s["dims"] = tuple(d)
    return s


def work_of(ops, case, states):
    """The case's work with the attended pairs of these inputs: their lanes have the case's lengths in another order, beside other
    counts of nodes."""
    w = dict(ops.work(case))
    if case["op"] == "attn" and case["ragged"]:
        counts, lens = ops._counts(case), [s["len"][s["slots"].long()].tolist() for s in states]
        pairs = lambda of: sum(n * x for n, x in zip(counts, of))  # noqa: E731
        w["flops"] += 4.0 * case["D"] * case["Hq"] * (statistics.mean(map(pairs, lens)) - pairs(ops._lens(case)))
    return w


def loop_us(run, passes, loops=5):
    """Microseconds of one call of run(k) among `passes` of them."""
    out = []
    for _ in range(loops):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for k in range(passes):
            run(k)
        b.record()
        b.synchronize()
        out.append(a.elapsed_time(b) * 1000 / passes)
    return statistics.median(out)


def rates():
    """Bytes per second of a large copy (read and written), operations per second of a large product, by type."""
    x = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)
    out = {"bytes": 2e6 * x.numel() / loop_us(lambda k: y.copy_(x), 20)}
    for name, dt in (("f32", torch.float32), ("bf16", torch.bfloat16), ("f16", torch.float16)):
        a, b = (torch.randn(8192, 8192, device="cuda", dtype=dt) for _ in range(2))
        out[name] = 2e6 * 8192 ** 3 / loop_us(lambda k: torch.mm(a, b), 100)
    return out


def error(got, want):
    """Distance of the floating outputs, the largest; whole numbers have to be equal."""
    worst = 0.0
    for name, w in want.items():
        if w is None:
            continue
        g = got[name].cpu()
        w = torch.as_tensor(w).cpu()
        if not g.is_floating_point():
            assert torch.equal(g.to(w.dtype), w), f"{name} differs"
        elif float(w.double().norm()) > 0:
            worst = max(worst, float((g.double() - w.double()).norm() / w.double().norm()))
    return worst


def kernel_of(name):
    """Name and template arguments of one of this library's kernels, else None; a profiler leaves the names with 16-bit types
    mangled."""
    m = re.search(r"\bgdn::.*?(\w+_kernel)(?:<([^>]*)>)?\(", name)
    if m:  # (a demangler that does not know bfloat16 takes it for another type, with the argument behind it)
        args = (m[2] or "").replace("bool _Accum, bool, E", "bf16, true").replace("bool _Accum", "bf16, float")
        return f"{m[1]}<{args}>" if args else m[1]
    m = re.match(r"_ZN3gdn12_GLOBAL__N_1\d+([a-z]\w*?_kernel)(?:I((?:DF16b|DF16_|f|Li\d+E|Lb[01]E)+)E)?", name)
    if not m:
        return None
    types = {"DF16b": "bf16", "DF16_": "f16", "f": "float", "Lb0E": "false", "Lb1E": "true"}
    args = [types.get(a) or a[2:-1] for a in re.findall(r"DF16b|DF16_|f|Li\d+E|Lb[01]E", m[2] or "")]
    return f"{m[1]}<{', '.join(args)}>" if args else m[1]


def by_case(path, value):
    """A profiler's CSV: for every case in order, the values of its kernels in the order of their first dispatch.  A case's
    dispatches follow each other; other kernels (the next one's inputs) lie between two cases."""
    rows = sorted(csv.DictReader(open(path, newline="")), key=lambda r: int(r["Dispatch_Id"]))
    out, inside = [], False
    for r in rows:
        name = kernel_of(r["Kernel_Name"])
        if name and not inside:
            out.append({})
        inside = name is not None
        if inside:
            out[-1].setdefault(name, []).append(value(r))
    return out


def summary(names, trace, fetch=None, write=None):
    """Markdown table of the cases' kernels."""
    us = by_case(trace, lambda r: (int(r["End_Timestamp"]) - int(r["Start_Timestamp"])) / 1e3)
    mb = [by_case(f, lambda r: float(r["Counter_Value"]) * 1024 / 1e6) for f in (fetch, write) if f]
    assert all(len(x) == len(names) for x in (us, *mb)), f"{[len(x) for x in (us, *mb)]} groups of dispatches, {len(names)} cases"
    lines = ["| case | kernel | us |" + (" read MB (counter) | written MB |" if len(mb) == 2 else ""), "|---|---|---|" + "---|---|" * (len(mb) == 2)]
    for k, name in enumerate(names):
        for kernel, times in us[k].items():
            cells = [name, kernel, f"{statistics.median(times):.1f}", *(f"{statistics.median(x[k][kernel]):.2f}" for x in mb)]
            lines.append("| " + " | ".join(cells) + " |")
            name = ""
    return "\n".join(lines)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--more", action="store_true", help="the cases of perf/more_operators.py")
    ap.add_argument("--only", default="", help="cases whose name holds this text")
    ap.add_argument("--further", action="store_true")
    ap.add_argument("--draw", type=int, default=0)
    ap.add_argument("--seed", type=int, default=0)
    ap.add_argument("--plain", action="store_true")
    ap.add_argument("--errors", action="store_true")
    ap.add_argument("--passes", type=int, default=0, help="passes of each case, one loop, without rates (for a profiler)")
    ap.add_argument("--summary", nargs="+", metavar="CSV")
    a = ap.parse_args(argv)
    ops = operators(a.more)
    if a.summary:
        print(summary([c["name"] for c in cases(ops, a.further, a.draw, a.seed, a.only)], *a.summary))
        return
    rate = None if a.passes else rates()
    if rate:
        print(f"copy {rate['bytes'] / 1e9:.0f} GB/s, products {', '.join(f'{k} {rate[k] / 1e12:.0f}' for k in DTYPES)} TFLOP/s", flush=True)
    for case in cases(ops, a.further, a.draw, a.seed, a.only):
        states = [prepare(ops, case, 1 + k) for k in range(3)]
        line = f"{case['name']:34s}"
        for own in ((False, True) if a.plain else (True,)):
            ops.own = own
            run = lambda k: ops.run(states[k % 3])  # noqa: E731
            for k in range(3):
                run(k)
            torch.cuda.synchronize()
            if a.passes:
                loop_us(run, a.passes, 1)
                continue
            once = loop_us(run, 3, 1)
            line += f" {'here' if own else 'plain':5s} {loop_us(run, max(5, min(300, int(3e5 / once)))):9.1f} us"
        if rate:
            w = work_of(ops, case, states)
            line += f"  floor {1e6 * max(w['bytes'] / rate['bytes'], w['flops'] / rate[case['dtype']]):7.1f} us"
        ops.own = True
        if a.errors:
            del states
            want = ops.exact({k: v for k, v in case.items() if k != "rows"}, 1)
            for own in (False, True):
                ops.own = own
                if want is not None:
                    line += f"  {'here' if own else 'plain'} off by {error(ops.run(prepare(ops, case, 1)), want):.1e}"
        if case["name"].startswith("draw"):
            line += f"  {({k: v for k, v in case.items() if k != 'name'})}"
        print(line, flush=True)
        states = None
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
