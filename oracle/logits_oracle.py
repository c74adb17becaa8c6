"""fp64 oracle of the call in gdn_logits.h, one row at a time.  It shares nothing with the HIP path."""

from __future__ import annotations

import numpy as np

from .round_oracle import LENGTH, NODES, PARENT, SLOT_RANGE, TOKEN, path_of

RULE = 512


def lane_bits(c, N, V, slot_ids, max_history, rules, tokens, parents, lane_nodes):
    """(bits, slot, nodes) of lane c; slot -1 is padding."""
    s, n = int(slot_ids[c]), N if lane_nodes is None else int(lane_nodes[c])
    if s == -1:
        return 0, -1, 0
    bits = 0 if 0 <= n <= N else NODES
    P = rules["P"]
    if not -1 <= s < P:
        bits |= SLOT_RANGE
    else:
        for name in ("repetition", "presence", "frequency", "temperature"):
            v = rules.get(name)
            if v is not None and (not np.isfinite(v[s]) or (name == "repetition" and not 2.0 ** -126 <= v[s] <= 2.0 ** 126) or (name == "temperature" and v[s] < 0)):
                bits |= RULE
        if rules.get("history") is not None:
            held = int(rules["history_len"][s])
            prompt = 0 if rules.get("prompt_len") is None else int(rules["prompt_len"][s])
            if not 0 <= held <= max_history or not 0 <= prompt <= held:
                bits |= LENGTH
    if not bits & NODES:
        if parents is not None and any(not -1 <= int(parents[c][i]) < i for i in range(n)):
            bits |= PARENT
        if tokens is not None and any(not 0 <= int(t) < V for t in tokens[c][:n]):
            bits |= TOKEN
    return bits, s, n


def adjusted(row, i, c, s, V, rules, mask, tokens, parents):
    """(z, what its size was before anything cancelled) of node i's row."""
    z = row.astype(np.float64).copy()
    size = np.abs(z)
    if rules.get("bias_tokens") is not None:
        for t, b in zip(rules["bias_tokens"][s], rules["bias"][s]):
            if 0 <= t < V:
                z[t] += float(b)
                size[t] += abs(float(b))
    seen, n = np.zeros(V, bool), np.zeros(V, np.int64)
    if rules.get("history") is not None:
        prompt = 0 if rules.get("prompt_len") is None else int(rules["prompt_len"][s])
        for at, t in enumerate(rules["history"][s][:int(rules["history_len"][s])]):
            if 0 <= t < V:
                seen[t] = True
                n[t] += at >= prompt
    if tokens is not None:
        for j in path_of(None if parents is None else parents[c], i):
            seen[tokens[c][j]] = True
            n[tokens[c][j]] += 1
    get = lambda name, other: other if rules.get(name) is None else float(rules[name][s])  # noqa: E731
    r, f, p = get("repetition", 1.0), get("frequency", 0.0), get("presence", 0.0)
    z = np.where(seen, np.where(z > 0, z / r, z * r), z)
    size = np.where(seen, size * max(r, 1 / r), size) + np.abs(f) * n + abs(p) * (n > 0)
    z = np.where(n > 0, z - f * n - p, z)
    if mask is not None:
        allowed = (mask[c, i].view(np.uint32)[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
        z = np.where(allowed == 1, z, -np.inf)
    return z, size


def probabilities(z, T):
    top = np.max(np.where(np.isnan(z), -np.inf, z))
    if T == 0:
        out = np.zeros(len(z))
        if top > -np.inf:
            out[int(np.nonzero(z == top)[0][0])] = 1.0
        return out
    if np.isnan(z).any():
        return np.full(len(z), np.nan)
    if top == -np.inf:
        return np.zeros(len(z))
    with np.errstate(invalid="ignore"):
        e = np.where(z == top, 1.0, np.exp((z - top) / T))
    return e / e.sum()


def adjust_logits(logits, slot_ids, rules, max_history, mask=None, tokens=None, parents=None, lane_nodes=None, rows=None):
    """({(c, i): (z, size, T or None)}, status); rules holds P and the arrays by name; rows: only these (c, i)."""
    C, N, V = logits.shape
    status, out = 0, {}
    for c in range(C):
        bits, s, n = lane_bits(c, N, V, slot_ids, max_history, rules, tokens, parents, lane_nodes)
        status |= bits
        if s == -1 or bits:
            continue
        for i in range(n):
            if rows is None or (c, i) in rows:
                z, size = adjusted(logits[c, i], i, c, s, V, rules, mask, tokens, parents)
                out[c, i] = (z, size, None if rules.get("temperature") is None else float(rules["temperature"][s]))
    return out, status
