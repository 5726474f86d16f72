"""Speculative decoding over the paged FP8 cache — oracle (numpy, float64).

Plain restatements of the calls of ``include/kvq_spec.h``: block tables as
Python lists, attention row by row over the tokens a row sees.
"""
from __future__ import annotations

import numpy as np

from . import fp8


def resize(table, held, target, block_tokens, free):
    """Block tables after a resize. ``table`` int [B, MB], ``free`` the list of
    free blocks (last on top). Returns (table, held, free, granted)."""
    table, free = np.array(table), list(free)
    held = [int(x) for x in held]
    width = table.shape[1]
    need = [-1 if t < 0 or -(-int(t) // block_tokens) > width else -(-int(t) // block_tokens) for t in target]
    released = []
    for b, n in enumerate(need):
        if 0 <= n < held[b]:
            released += table[b, n:held[b]].tolist()
            table[b, n:held[b]] = -1
            held[b] = n
    free += released[::-1]
    granted, asked, room = [], 0, len(free)
    for b, n in enumerate(need):
        grow = max(0, n - held[b])
        asked += grow
        ok = n >= 0 and (grow == 0 or asked <= room)
        granted.append(int(ok))
        if ok:
            for j in range(held[b], held[b] + grow):
                table[b, j] = free.pop()
            held[b] += grow
    return table, np.array(held, np.int32), free, np.array(granted, np.int32)


def slot_map(table, seq_lens, new_lens, block_tokens, num_blocks, rows):
    """(offsets [B+1], slots, seq_ids, positions) of the new tokens, rows behind them -1."""
    slots, seqs, poss, offsets = [], [], [], [0]
    width = table.shape[1]
    for b, (n0, n) in enumerate(zip(seq_lens, new_lens)):
        for p in range(int(n0), int(n0) + max(0, int(n))):
            if len(slots) == rows:
                break
            inside = 0 <= p < min(width * block_tokens, 2**31)
            blk = int(table[b, p // block_tokens]) if inside else -1
            slots.append(blk * block_tokens + p % block_tokens if 0 <= blk < num_blocks else -1)
            seqs.append(b)
            poss.append(p if p < 2**31 else -1)
        offsets.append(len(slots))
    pad = [-1] * (rows - len(slots))
    return (np.array(offsets, np.int32), np.array(slots + pad, np.int64), np.array(seqs + pad, np.int32),
            np.array(poss + pad, np.int32))


def append(pool, x16, slots, scale, fmt):
    """Natural pool bytes [nb, H, 16, D] with tokens x16 [N, H, D] quantized into the rows of ``slots``."""
    out = pool.copy()
    byte = fp8.quantize(x16.transpose(1, 0, 2)[None], scale, fmt)[0].transpose(1, 0, 2)
    for i, s in enumerate(slots):
        if 0 <= s < pool.shape[0] * 16:
            out[s // 16, :, s % 16] = byte[i]
    return out


def accept(pool, table, seq_lens, path, n_accepted):
    """Natural pool bytes with each request's accepted rows moved to the end of its sequence."""
    out = pool.copy()
    for b, n in enumerate(n_accepted):
        for i in range(int(n)):
            p, q = int(seq_lens[b]) + int(path[b][i]), int(seq_lens[b]) + i
            out[table[b, q // 16], :, q % 16] = pool[table[b, p // 16], :, p % 16]
    return out


def tree_attention(q16, k_pool, v_pool, k_scale, v_scale, fmt, table, seq_lens, offsets, sees, scale):
    """Float64 tree attention over natural pools [nb, H, 16, D]: ``sees`` is a
    boolean [N, nodes]. Returns (out, mag, spread, dots), each [N, Hq, D] or
    [N, Hq]: the output, the same sum over |v|, the sum of |v| over the seen
    tokens divided by the softmax's sum, and the largest sum of |q k| * scale."""
    n, hq, d = q16.shape
    h = k_pool.shape[1]
    gq = hq // h
    ks, vs = np.broadcast_to(k_scale, (h,)).astype(np.float64), np.broadcast_to(v_scale, (h,)).astype(np.float64)
    out, mag, spread = (np.zeros((n, hq, d)) for _ in range(3))
    dots = np.zeros((n, hq))
    for b in range(len(seq_lens)):
        ctx, n0, n1 = int(seq_lens[b]), int(offsets[b]), int(offsets[b + 1])
        total = ctx + n1 - n0
        if n1 == n0 or total == 0:
            continue
        rows = np.arange(total)
        blk = table[b, rows // 16]
        for hi in range(h):
            with np.errstate(invalid="ignore"):
                kk = fp8.decode(k_pool[blk, hi, rows % 16], fmt) * ks[hi]
                vv = fp8.decode(v_pool[blk, hi, rows % 16], fmt) * vs[hi]
            for i in range(n0, n1):
                vis = np.concatenate([np.ones(ctx, bool), sees[i, : n1 - n0]])
                if not vis.any():
                    continue
                k1, v1 = kk[vis], vv[vis]
                for g in range(hi * gq, (hi + 1) * gq):
                    q = q16[i, g].astype(np.float64)
                    s = k1 @ q * float(scale)
                    p = np.exp(s - s.max())
                    out[i, g] = p @ v1 / p.sum()
                    mag[i, g] = p @ np.abs(v1) / p.sum()
                    spread[i, g] = np.abs(v1).sum(0) / p.sum()
                    dots[i, g] = (np.abs(k1) @ np.abs(q)).max() * float(scale)
    return out, mag, spread, dots
