"""What the operators on pages (kv_fork, kv_compact) do, in plain loops over
rows and pages, from their definitions in include/sv.h; and the 64-bit form of
the log probabilities."""
from __future__ import annotations

import numpy as np

PAGE = 16


def fork(table, length, held, refs, source=None, keep=None, room=None):
    """(table, length, held, refs, moves), or None where nothing changes."""
    S, W = table.shape
    source = list(range(S)) if source is None else list(source)
    refs = [int(x) for x in refs]
    rows, sizes, needs = [], [], []
    for s in range(S):
        a = source[s]
        if a < -1 or a >= S:
            return None
        if a < 0:
            rows.append([]), sizes.append(0), needs.append(0)
            continue
        n = min(int(length[a]), int(held[a]) * PAGE, 1 << 30 if keep is None else max(0, int(keep[s])))
        rows.append([int(x) for x in table[a][:-(-n // PAGE)]])
        sizes.append(n)
        needs.append(max(len(rows[-1]), -(-max(0, 0 if room is None else int(room[s])) // PAGE)))
        if needs[-1] > W:
            return None
    for s in range(S):
        for p in table[s][:held[s]]:
            if 0 <= p < len(refs):
                refs[p] -= 1
    for row in rows:
        for p in row:
            if 0 <= p < len(refs):
                refs[p] += 1
    begun = {}
    for s in range(S):
        if sizes[s] % PAGE and 0 <= rows[s][-1] < len(refs):
            begun.setdefault(rows[s][-1], []).append(s)
    copies = set()
    for p, holders in begun.items():
        if refs[p] > 1:
            copies |= set(holders[1:] if refs[p] == len(holders) else holders)
    for s in copies:
        refs[rows[s][-1]] -= 1
    free = [p for p, n in enumerate(refs) if n == 0]
    if sum(needs[s] - len(rows[s]) + (s in copies) for s in range(S)) > len(free):
        return None
    moves = np.full((S, 2), -1)
    take = iter(free)
    for s in range(S):
        if s in copies:
            moves[s] = rows[s][-1], next(take)
            rows[s][-1] = moves[s][1]
            refs[moves[s][1]] = 1
        while len(rows[s]) < needs[s]:
            rows[s].append(next(take))
            refs[rows[s][-1]] = 1
    out = np.full((S, W), -1)
    for s in range(S):
        out[s, :len(rows[s])] = rows[s]
    return out, np.array(sizes), np.array(needs), np.array(refs), moves


def compact(table, length, held, refs, most):
    """(table, refs, moves, where)."""
    used = [p for p in range(len(refs)) if refs[p] > 0][::-1]
    free = [p for p in range(len(refs)) if refs[p] == 0]
    pairs = [(a, b) for a, b in zip(used, free) if a > b][:most]
    where = np.array([p if refs[p] else -1 for p in range(len(refs))])
    refs = np.array(refs)
    for a, b in pairs:
        where[a] = b
        refs[b], refs[a] = refs[a], 0
    out = np.full(table.shape, -1)
    for s in range(table.shape[0]):
        for j in range(held[s]):
            out[s, j] = where[table[s, j]]
    moves = np.full((most, 2), -1)
    moves[:len(pairs)] = np.array(pairs).reshape(-1, 2)
    return out, refs, moves, where


def logprobs(x, tokens, scale, top):
    """x: float64 [n, vocab]. (out, lse, entropy, top_values, top_ids), NaN and -1 for rows without a distribution."""
    n, vocab = x.shape
    y = x * np.float64(np.float32(scale))
    out, lse, ent = np.zeros(tokens.shape), np.full(n, np.nan), np.full(n, np.nan)
    tv, ti = np.full((n, top), np.nan), np.full((n, top), -1)
    for r in range(n):
        good = not np.isnan(y[r]).any() and not (y[r] == np.inf).any() and (y[r] > -np.inf).any()
        if good:
            m = y[r].max()
            w = np.exp(y[r] - m)
            lse[r] = m + np.log(w.sum())
            p = w / w.sum()
            lp = (y[r] - m) - np.log(w.sum())  # (y - lse would lose the sum beside logits of 1e17 and more)
            ent[r] = -(p[p > 0] * lp[p > 0]).sum()
            order = np.lexsort((np.arange(vocab), -x[r]))[:top]
            order = order[x[r][order] > -np.inf]
            tv[r] = -np.inf
            tv[r, :len(order)], ti[r, :len(order)] = lp[order], order
        for i, t in enumerate(tokens[r]):
            out[r, i] = 0.0 if t == -1 else np.nan if not good or not 0 <= t < vocab else lp[t]
    return out, lse, ent, tv, ti
