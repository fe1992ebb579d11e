"""Float64 reference of one speculative decoding step: attention of drafted
trees, verification of the drafted tokens, compaction of the cache."""
from __future__ import annotations

import numpy as np


def ancestors(parents, row):
    """Rows on the way up from `row`, itself first."""
    way = []
    while row >= 0:
        way.append(row)
        row = int(parents[row])
    return way


def tree_mask(parents, ctx, n_keys, window_left=-1):
    """[rows, keys] visibility of one request's keys for its rows."""
    n = len(parents)
    seen = np.zeros((n, n_keys), dtype=bool)
    for i in range(n):
        way = ancestors(parents, i)
        pos = ctx + len(way) - 1
        for j in range(min(max(ctx, 0), n_keys)):
            seen[i, j] = window_left < 0 or j >= pos - window_left
        for far, a in enumerate(way):
            if 0 <= ctx + a < n_keys and (window_left < 0 or
                                          far <= window_left):
                seen[i, ctx + a] = True
    return seen


def tree_attention(q, k, v, parents, scale, softcap=0.0, window_left=-1,
                   sinks=None):
    """One request: q [n, Hq, D], k / v [L, Hkv, D]; out [n, Hq, D] and lse
    [Hq, n]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    n_keys, hkv = k.shape[0], k.shape[1]
    seen = tree_mask(parents, n_keys - n, n_keys, window_left)
    out = np.zeros((n, hq, d))
    lse = np.full((hq, n), -np.inf)
    for h in range(hq):
        kh, vh = k[:, h // (hq // hkv)], v[:, h // (hq // hkv)]
        for i in range(n):
            x = scale * (kh[seen[i]] @ q[i, h])
            if softcap > 0:
                x = softcap * np.tanh(x / softcap)
            z = x if sinks is None else np.append(x, sinks[h])
            if z.size == 0:
                continue
            top = z.max()
            total = np.exp(z - top).sum()
            lse[h, i] = top + np.log(total)
            out[i, h] = np.exp(x - lse[h, i]) @ vh[seen[i]]
    return out, lse


def verify(target, tokens, uniform, parents, draft=None):
    """One request's rows: (tokens said, rows that stand)."""
    target = np.asarray(target, np.float64)
    # (probabilities below 0 or NaN count as 0)
    draft = None if draft is None else \
        np.fmax(np.asarray(draft, np.float64), 0.0)
    n, vocab = target.shape
    node, said, rows = 0, [], [0]
    rest, mass = np.maximum(target[0], 0.0), 1.0
    for i in range(1, n):
        if parents[i] != node:
            continue
        x = int(tokens[i])
        if not 0 <= x < vocab:
            continue
        likely = 1.0 if draft is None else draft[node, x]
        if float(uniform[i]) * likely * mass < rest[x]:
            node = i
            said.append(x)
            rows.append(i)
            rest, mass = np.maximum(target[i], 0.0), 1.0
        elif draft is None:
            mass = max(mass - rest[x], 0.0)
            rest[x] = 0.0
        else:
            rest = np.maximum(rest - mass * draft[node], 0.0)
            mass = rest.sum()
    if not rest.sum() > 0:
        rest = np.maximum(target[node], 0.0)
    run = np.cumsum(rest)
    over = np.flatnonzero(run > float(uniform[0]) * run[-1])
    some = np.flatnonzero(rest > 0)
    said.append(int(over[0] if over.size else some[-1] if some.size else -1))
    return said, rows


def compact(cache, table, ctx, rows):
    """cache [NB, BS, ...] of one request with its rows moved together."""
    bs = cache.shape[1]
    out = cache.copy()
    for i, r in enumerate(rows):
        to, of = ctx + i, ctx + int(r)
        out[table[to // bs], to % bs] = cache[table[of // bs], of % bs]
    return out
