"""fp64 oracle of the calls in gdn_round.h, one lane / node / head at a time.

It evaluates the plain definitions with numpy in float64 and shares nothing with the HIP path.
Lanes that the calls skip (padding, an error bit) are left out of the results; the status bits
are returned beside them.
"""

from __future__ import annotations

import numpy as np

SLOT_RANGE, SLOT_DUP, PARENT, ACCEPT, NODES, LENGTH, PAGE, TOKEN, AXIS = 1, 2, 4, 8, 16, 32, 64, 128, 256


def path_of(parents, i):
    """Nodes from the prefix's child down to i; parents None: a chain."""
    if parents is None:
        return list(range(i + 1))
    out = []
    while i >= 0:
        out.append(int(i))
        i = int(parents[i])
    return out[::-1]


def parent_list(parents, n):
    return [i - 1 for i in range(n)] if parents is None else [int(p) for p in parents[:n]]


def lane_bits(c, N, slot_ids, seq_len, capacity, parents, lane_nodes, dup=False):
    """(bits, slot, nodes, length) of lane c; slot -1 is padding."""
    s, n = int(slot_ids[c]), N if lane_nodes is None else int(lane_nodes[c])
    if s == -1:
        return 0, -1, 0, 0
    bits, length = 0, 0
    if n < 0 or n > N:
        bits |= NODES
    if s < -1 or s >= len(seq_len):
        bits |= SLOT_RANGE
    else:
        length = int(seq_len[s])
        if length < 0 or length + max(n, 0) > capacity:
            bits |= LENGTH
        if dup and sum(int(o) == s for o in slot_ids) > 1:
            bits |= SLOT_DUP
    if parents is not None and not bits & NODES:
        if any(not -1 <= int(parents[c][i]) < i for i in range(n)):
            bits |= PARENT
    return bits, s, n, length


def rms_norm(x, w, eps):
    return x if w is None else x / np.sqrt(np.mean(x * x) + eps) * w


def rotate(x, angles, interleaved):
    """Turns pair j of the first 2 * len(angles) values by angles[j]."""
    half = len(angles)
    y = np.array(x, np.float64)
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        co, si = np.cos(angles[j]), np.sin(angles[j])
        y[a], y[b] = x[a] * co - x[b] * si, x[b] * co + x[a] * si
    return y


def rope_kv_write(q, k, v, inv_freq, k_cache, v_cache, slot_ids, page_table, seq_len, positions=None, pair_axis=None,
                  parents=None, lane_nodes=None, q_norm=None, k_norm=None, eps=1e-6, interleaved=False, n_axes=1):
    """Writes into k_cache, v_cache (float64) in place; returns ({(c, i): q rows}, status)."""
    C, N, Hq, D = q.shape
    Hkv, page = k_cache.shape[1], k_cache.shape[2]
    status, out = 0, {}
    axes = np.zeros(len(inv_freq), int) if pair_axis is None else np.asarray(pair_axis)
    for c in range(C):
        bits, s, n, length = lane_bits(c, N, slot_ids, seq_len, page_table.shape[1] * page, parents, lane_nodes, dup=True)
        if s == -1:
            continue
        if ((axes < 0) | (axes >= n_axes)).any():
            bits |= AXIS
        if bits:
            status |= bits
            continue
        for i in range(n):
            depth = len(path_of(None if parents is None else parents[c], i)) - 1
            pos = np.full(len(axes), length + depth, np.float64) if positions is None else positions[c, i, axes].astype(np.float64)
            ang = pos * np.asarray(inv_freq, np.float64)
            out[c, i] = np.stack([rotate(rms_norm(q[c, i, h].astype(np.float64), q_norm, eps), ang, interleaved)
                                  for h in range(Hq)])
            pid = int(page_table[s, (length + i) // page])
            if not 0 <= pid < k_cache.shape[0]:
                status |= PAGE
                continue
            for h in range(Hkv):
                k_cache[pid, h, (length + i) % page] = rotate(rms_norm(k[c, i, h].astype(np.float64), k_norm, eps), ang, interleaved)
                v_cache[pid, h, (length + i) % page] = v[c, i, h]
    return out, status


def silu_or_sigmoid(z, mode):
    sig = 1.0 / (1.0 + np.exp(-z))
    return z * sig if mode == 0 else sig


def paged_attention(q, k_cache, v_cache, slot_ids, page_table, seq_len, parents=None, lane_nodes=None, scale=None,
                    gate=None, gate_mode=1):
    """Returns ({(c, i): (out [Hq, D], weighted |V| [Hq, D], largest |q||k| sum, rows)}, status)."""
    C, N, Hq, D = q.shape
    n_pages, Hkv, page, _ = k_cache.shape
    G, scale = Hq // Hkv, D ** -0.5 if scale is None else scale
    status, res = 0, {}
    for c in range(C):
        bits, s, n, length = lane_bits(c, N, slot_ids, seq_len, page_table.shape[1] * page, parents, lane_nodes)
        if s == -1 or bits:
            status |= bits
            continue
        for i in range(n):
            want = list(range(length)) + [length + j for j in path_of(None if parents is None else parents[c], i)]
            rows = []
            for t in want:
                pid = int(page_table[s, t // page])
                if 0 <= pid < n_pages:
                    rows.append((pid, t % page))
                else:
                    status |= PAGE
            out, mag, big = np.zeros((Hq, D)), np.zeros((Hq, D)), 0.0
            for h in range(Hq):
                if not rows:
                    continue
                pids, at = np.array(rows).T
                kk, vv = k_cache[pids, h // G, at].astype(np.float64), v_cache[pids, h // G, at].astype(np.float64)
                x = kk @ q[c, i, h].astype(np.float64) * scale
                big = max(big, float(np.max(np.abs(kk) @ np.abs(q[c, i, h].astype(np.float64)))) * scale)
                w = np.exp(x - x.max())
                out[h], mag[h] = w @ vv / w.sum(), w @ np.abs(vv) / w.sum()
            if gate is not None:
                act = silu_or_sigmoid(gate[c, i].astype(np.float64), gate_mode)
                out, mag = out * act, mag * np.abs(act)
            res[c, i] = (out, mag, big, len(rows))
    return res, status


def draw(w, u):
    """The lowest index whose running sum exceeds u times the whole; -1 without weight."""
    total = np.cumsum(w)
    if not total[-1] > 0:
        return -1
    over = np.nonzero((total > u * total[-1]) & (w > 0))[0]
    return int(over[0]) if len(over) else int(np.nonzero(w)[0][-1])


def largest(row):
    """Index of the largest value, the lowest of equal ones; NaN below all, minus infinity among them."""
    known = np.nonzero(~np.isnan(row))[0]
    return int(known[np.argmax(row[known])]) if len(known) else 0


def draft_accept(target, tokens, root=None, draft=None, parents=None, lane_nodes=None, slot_ids=None, u_accept=None,
                 u_next=None):
    """Returns ({c: (accept_node, n_accept, next_token)}, status)."""
    C, N, V = target.shape
    status, res = 0, {}
    for c in range(C):
        if slot_ids is not None and slot_ids[c] == -1:
            continue
        n, bits = N if lane_nodes is None else int(lane_nodes[c]), 0
        if n < 0 or n > N:
            bits |= NODES
        else:
            if any(not 0 <= int(t) < V for t in tokens[c][:n]):
                bits |= TOKEN
            if parents is not None and any(not -1 <= int(parents[c][i]) < i for i in range(n)):
                bits |= PARENT
        if bits:
            status |= bits
            continue
        par = parent_list(None if parents is None else parents[c], n)
        node, count = -1, 0
        while True:
            row = target[c, node] if node >= 0 else None if root is None else root[c]
            p = None if row is None else np.where(row.astype(np.float64) > 0, row.astype(np.float64), 0.0)
            best = None if row is None else largest(row)
            refused, went, left = [], None, 1.0
            kids = [j for j in range(n) if par[j] == node]
            for j in kids:
                t = int(tokens[c][j])
                if row is None:
                    went = j
                elif t in refused:
                    continue
                elif u_accept is None:
                    went = j if t == best else None
                else:
                    qq = 1.0 if draft is None else max(float(draft[c, j, t]), 0.0)
                    if float(u_accept[c, j]) * qq * left < p[t]:
                        went = j
                if went is not None:
                    break
                refused.append(t)
                left -= p[t] if p is not None else 0.0
            if went is None:
                break
            node, count = went, count + 1
        if row is None:
            token = -1
        elif u_accept is None:
            token = best
        else:
            w = p.copy()
            if draft is not None and kids:
                qd = draft[c, kids[0]].astype(np.float64)
                w = np.maximum(p - np.where(qd > 0, qd, 0.0), 0.0)
            elif refused:
                w[refused] = 0.0
            token = draw(w if w.sum() > 0 else p, float(u_next[c]))
        res[c] = (node, count, token)
    return res, status


def kv_commit(k_caches, v_caches, slot_ids, page_table, seq_len, accept_node, parents=None, lane_nodes=None, status_in=0, N=None):
    """Moves rows of the given arrays in place and returns (new_len, status)."""
    C = len(slot_ids)
    N = N if parents is None else len(parents[0])
    page, n_pages = k_caches[0].shape[2], k_caches[0].shape[0]
    bits = 0
    for c in range(C):
        b, s, n, length = lane_bits(c, N, slot_ids, seq_len, page_table.shape[1] * page, parents, lane_nodes, dup=True)
        bits |= b
        if s == -1:
            continue
        if not -1 <= int(accept_node[c]) < min(max(n, 0), N):
            bits |= ACCEPT
        if parents is not None and not b & ~(PARENT | SLOT_DUP):
            for i in range(n):
                if not 0 <= int(page_table[s, (length + i) // page]) < n_pages:
                    bits |= PAGE
    new_len = np.array(seq_len, np.int32)
    if bits or status_in:
        return new_len, bits | status_in
    for c in range(C):
        s, e = int(slot_ids[c]), int(accept_node[c])
        if s == -1 or e < 0:
            continue
        path, length = path_of(None if parents is None else parents[c], e), int(seq_len[s])
        for j, a in enumerate(path):
            (dp, do), (sp, so) = divmod(length + j, page), divmod(length + a, page)
            for t in (*k_caches, *v_caches):
                if (dp, do) != (sp, so):
                    t[int(page_table[s, dp]), :, do] = t[int(page_table[s, sp]), :, so]
        new_len[s] = length + len(path)
    return new_len, bits
