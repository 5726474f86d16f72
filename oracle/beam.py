"""Beam search over the paged FP8 cache — oracle (numpy, float64).

Plain restatements of the calls of ``include/kvq_beam.h``: block tables as
Python lists, candidates by a full sort, attention sequence by sequence.
"""
from __future__ import annotations

import numpy as np

from . import spec


def select(logits, scores, n_out, finished=None, end_token=-1):
    """(scores float64, parents, tokens), each [R, n_out], of logits [R * W, V] and scores [R, W]."""
    r, w = scores.shape
    v = logits.shape[1]
    big = float(np.finfo(np.float32).max)
    out = []
    for g in range(r):
        total = np.full((w, v), -np.inf)
        for i in range(w):
            s = float(scores[g, i])
            if finished is not None and finished[g, i]:
                total[i, end_token] = s if np.isfinite(s) else -np.inf
                continue
            x = logits[g * w + i].astype(np.float64)
            x = np.minimum(np.where(np.isnan(x), -np.inf, x), big)
            if not np.isfinite(s) or x.max() == -np.inf:
                continue
            d = x - x.max()
            total[i] = s + (d - np.log(np.exp(d).sum()))
        flat = total.reshape(-1)
        order = np.lexsort((np.arange(w * v), -flat))[:n_out]
        out.append((flat[order], order // v, order % v))
    return tuple(np.array([o[k] for o in out]) for k in range(3))


def fork(table, held, lens, parents, width, block_tokens, shares, free):
    """The tables after every sequence has become a copy of its parent: a dict of table, held, lens, shares, free (the
    list of free blocks, last on top), pairs (of blocks to copy), granted and shared (leading blocks of each request)."""
    table, shares, free = np.array(table), list(map(int, shares)), list(map(int, free))
    b, most = table.shape
    blocks = len(shares)
    held = [min(max(int(h), 0), most) for h in held]
    lens = [min(max(int(n), 0), h * block_tokens) for n, h in zip(lens, held)]
    rows, new_lens = [], []
    for i, p in enumerate(parents):
        p = int(p)
        src = i // width * width + p
        n = lens[src] if 0 <= p < width else 0
        rows.append(table[src, : -(-n // block_tokens)].tolist() if n else [])
        new_lens.append(n)
    refs = {}
    for row in rows:
        for x in row:
            refs[x] = refs.get(x, 0) + 1
    for i in range(b):
        for x in table[i, : held[i]].tolist():
            refs[x] = refs.get(x, 0) - 1
    freed = []
    for x, change in refs.items():
        if 0 <= x < blocks:
            shares[x] += change
            if shares[x] < 0:
                shares[x] = 0
                freed.append(x)
    free += sorted(freed, reverse=True)
    tails = [row[-1] if n % block_tokens and 0 <= row[-1] < blocks else None for row, n in zip(rows, new_lens)]
    pairs, granted, dropped = [], [], []
    for i, x in enumerate(tails):
        ok = 1
        if x is not None:
            mates = [j for j in range(i // width * width, i // width * width + width) if tails[j] == x]
            if not (shares[x] + 1 == len(mates) and mates[0] == i):
                ok = int(len(free) > 0)
                if ok:
                    rows[i][-1] = free.pop()
                    pairs.append((x, rows[i][-1]))
                    dropped.append(x)
        granted.append(ok)
    for x in dropped:
        shares[x] -= 1
    shared = []
    for g in range(b // width):
        live = [j for j in range(g * width, g * width + width) if new_lens[j] > 0]
        n = 0
        while live and all(new_lens[j] >= (n + 1) * block_tokens and rows[j][n] == rows[live[0]][n] for j in live):
            n += 1
        shared.append(n)
    for i in range(b):
        old = held[i]
        table[i, : max(old, len(rows[i]))] = -1
        table[i, : len(rows[i])] = rows[i]
    return dict(table=table, held=[len(x) for x in rows], lens=new_lens, shares=shares, free=free, pairs=pairs,
                granted=granted, shared=shared)


def compact(table, held, keep, shares, free, max_copies):
    """The tables after the blocks from keep on have been emptied: a dict of table, shares, free, pairs, moved_to, done."""
    table, shares, free = np.array(table), list(map(int, shares)), list(map(int, free))
    blocks = len(shares)
    empty = set(free)
    movers = [x for x in range(keep, blocks) if x not in empty]
    targets = [x for x in range(keep) if x in empty]
    moved = list(range(blocks))
    if len(movers) > len(targets) or len(movers) > max_copies:
        return dict(table=table, shares=shares, free=free, pairs=[], moved_to=moved, done=0)
    pairs = list(zip(movers, targets))
    for x, y in pairs:
        moved[x] = y
        shares[y], shares[x] = shares[x], 0
    for i in range(table.shape[0]):
        for j in range(int(held[i])):
            if 0 <= table[i, j] < blocks:
                table[i, j] = moved[table[i, j]]
    return dict(table=table, shares=shares, free=targets[len(movers):][::-1], pairs=pairs, moved_to=moved, done=1)


def group_attention(q16, k_pool, v_pool, k_scale, v_scale, fmt, table, seq_lens, scale):
    """Float64 decode attention over natural pools [nb, H, 16, D], sequence by sequence: each one's last token is a tree of
    one node behind the others. Returns what spec.tree_attention returns; zeros for an empty sequence."""
    n = len(seq_lens)
    outs = [np.zeros(q16.shape) for _ in range(3)] + [np.zeros(q16.shape[:2])]
    live = [b for b in range(n) if seq_lens[b] > 0]
    if live:
        got = spec.tree_attention(q16[live], k_pool, v_pool, k_scale, v_scale, fmt, np.asarray(table)[live],
                                  [int(seq_lens[b]) - 1 for b in live], np.arange(len(live) + 1),
                                  np.ones((len(live), 1), bool), scale)
        for o, g in zip(outs, got):
            o[live] = g
    return tuple(outs)
