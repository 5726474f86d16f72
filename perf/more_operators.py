"""Performance cases of beam search over the paged FP8 cache.

One step of a serving loop that keeps several continuations of each request:
the best candidates are selected from the logits, the block tables follow the
parents (blocks are shared, a partly filled last one is copied), the copies are
carried out in every layer's pools, the new tokens attend over the cache with
the blocks that a request's beams share read once. Now and then the pool is
compacted, so that its end can be given back. Each case is one of these
operators at a size such a loop meets. `run` computes it in elementary torch
operations, or with `own` through the library.
"""
import math

import torch

own = False

BT = 16                      # tokens of a pool block
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FLOAT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- cases

def _select(name, groups, width, vocab, out, dtype, banned, finished):
    """`out` candidates a request; `banned`: share of the tokens at -inf; `finished`: some beams have ended."""
    return {"name": name, "op": "select", "groups": groups, "width": width, "vocab": vocab, "out": out, "dtype": dtype,
            "banned": banned, "finished": finished}


def _fork(name, groups, width, shared_lo, shared_hi, own_hi, dropped):
    """Requests whose beams share shared_lo .. shared_hi blocks and hold up to own_hi tokens of their own; `dropped`:
    some requests end."""
    return {"name": name, "op": "fork", "groups": groups, "width": width, "shared_lo": shared_lo,
            "shared_hi": shared_hi, "own_hi": own_hi, "dropped": dropped}


def _copy(name, buffers, block_bytes, blocks, pairs):
    return {"name": name, "op": "copy", "buffers": buffers, "block_bytes": block_bytes, "blocks": blocks, "pairs": pairs}


def _compact(name, batch, held_lo, held_hi, blocks, keep):
    """A pool of `blocks` blocks, of which the requests hold held_lo .. held_hi each, is to end at block `keep`."""
    return {"name": name, "op": "compact", "batch": batch, "held_lo": held_lo, "held_hi": held_hi, "blocks": blocks,
            "keep": keep}


def _attend(name, groups, width, heads, q_heads, dim, shared_lo, shared_hi, own_lo, own_hi, fmt="e4m3", per_head=False):
    """Requests whose `width` beams share shared_lo .. shared_hi blocks and hold own_lo .. own_hi tokens each behind."""
    return {"name": name, "op": "attend", "groups": groups, "width": width, "heads": heads, "q_heads": q_heads,
            "dim": dim, "shared_lo": shared_lo, "shared_hi": shared_hi, "own_lo": own_lo, "own_hi": own_hi, "fmt": fmt,
            "per_head": per_head}


def listed():
    return [
        # one request's 4 beams, latency bound
        _select("select_1x4_v32000", 1, 4, 32000, 4, "fp32", 0.0, False),
        # an odd vocabulary (rows that start anywhere), banned tokens, beams that have ended, twice as many candidates
        _select("select_8x5_v50021", 8, 5, 50021, 10, "fp16", 0.01, True),
        # a full server: 512 rows of a large vocabulary
        _select("select_64x8_v128000", 64, 8, 128000, 16, "bf16", 0.0, True),
        # a small server's step over contexts of some 1000 tokens
        _fork("fork_8x4_1k", 8, 4, 20, 100, 200, False),
        # 512 beams over contexts of up to 32K tokens, some requests ending
        _fork("fork_64x8_32k", 64, 8, 100, 2000, 700, True),
        # the copies of a small step in the pools (keys and values) of 2 layers, latency bound
        _copy("copy_4_16k", 4, 16384, 512, 4),
        # those of a full server in 16 layers
        _copy("copy_448_16k", 32, 16384, 4096, 448),
        # a small pool, a quarter given back
        _compact("compact_8_4k", 8, 20, 120, 4096, 3001),
        # a large pool, half of it given back
        _compact("compact_512_1m", 512, 200, 1500, 1 << 20, 1 << 19),
        # one request's 4 beams over 1000 tokens, latency bound
        _attend("attend_1x4_s1000", 1, 4, 8, 32, 128, 62, 62, 1, 40),
        # several samples of each prompt, lengths of all kinds, 64 channels, E5M2 with a scale per head
        _attend("attend_16x5_ragged", 16, 5, 8, 16, 64, 30, 1024, 1, 3000, "e5m2", True),
        # 8 beams over the 128K cache, 8 query heads a kv head
        _attend("attend_4x8_s131072", 4, 8, 8, 64, 128, 8192, 8192, 20, 300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "fork", "copy", "compact", "attend", "attend"])
    width = _log(rng, 1, 16)
    if op == "select":
        vocab = _log(rng, 500, 160000)
        groups = max(1, min(_log(rng, 1, 200), 50_000_000 // (width * vocab)))
        dtype = rng.choice(["fp32", "fp16", "bf16"])
        if dtype == "fp32":
            groups = max(1, groups // 2)
        c = _select("", groups, width, vocab, rng.choice([1, width, 2 * width]), dtype,
                    rng.choice([0.0, 0.0, 0.02, 0.9]), rng.random() < 0.5)
    elif op == "fork":
        groups = max(1, _log(rng, 1, 400) // width)
        lo = _log(rng, 1, 1000) - 1
        c = _fork("", groups, width, lo, lo + _log(rng, 1, 1000), _log(rng, 1, 700), rng.random() < 0.5)
    elif op == "copy":
        size = 16 * _log(rng, 16, 2048)
        buffers = _log(rng, 1, 64)
        pairs = max(1, min(_log(rng, 1, 1500), 230_000_000 // (size * buffers)))
        blocks = 2 * pairs + rng.randrange(200)
        buffers = max(1, min(buffers, 2_000_000_000 // (blocks * size)))
        c = _copy("", buffers, size, blocks, pairs)
    elif op == "compact":
        batch, lo = _log(rng, 1, 400), _log(rng, 1, 500)
        hi = lo + _log(rng, 1, 1000)
        held = batch * (lo + hi) // 2 + batch
        blocks = int(held * rng.uniform(1.2, 4.0)) + 10
        c = _compact("", batch, lo, hi, blocks, rng.randint(held + 1, blocks))
    else:
        heads, gq, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        lo = _log(rng, 1, 6000) - 1
        hi = lo + _log(rng, 1, 1500)
        own_hi = _log(rng, 1, 4000)
        tokens = 16 * hi + width * own_hi
        # no more bytes and no more products than the largest listed case
        groups = max(1, min(_log(rng, 1, 64), 4 * 8 * 131072 * 128 // (tokens * heads * dim),
                            4 * 64 * 8 * 131072 * 128 // (width * heads * gq * (16 * hi + own_hi) * dim)))
        c = _attend("", groups, width, heads, heads * gq, dim, lo, hi, max(1, own_hi // _log(rng, 1, 100)), own_hi,
                    rng.choice(["e4m3", "e5m2"]), rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _spread(gen, lo, hi, n):
    """n whole numbers spread evenly over lo .. hi, in a random order: their sum goes by the case alone."""
    x = torch.arange(n) * (hi - lo) // max(1, n - 1) + lo if n > 1 else torch.tensor([hi])
    return x[torch.randperm(n, generator=gen)]


def _order(dim, role, device="cuda"):
    """Byte of (token row, channel) in a pool block of 16 x dim: int64 [16, dim]."""
    t, c = torch.arange(BT, device=device)[:, None], torch.arange(dim, device=device)[None, :]
    if role == "k":
        word = (t // 8) * (dim // 64) * 32 + c // 64 * 32 + 4 * (t % 8) + c % 16 // 4
        return word * 16 + c % 64 // 16 * 4 + c % 4
    return (c // 32 * 32 + 4 * (c % 8) + t % 8 // 2) * 16 + c % 32 // 8 * 4 + t // 8 * 2 + t % 2


def _random_pool(blocks, heads, dim, fmt, role, size, gen):
    """Pool bytes [blocks, heads, 16 * dim] of normal values, channel c of head h of size size[h, c]."""
    pool = torch.empty((blocks, heads, BT * dim), dtype=torch.uint8, device="cuda")
    width = torch.empty((heads, BT * dim), device="cuda")
    width[:, _order(dim, role).reshape(-1)] = size.repeat(1, BT)
    step = max(1, (1 << 26) // (heads * BT * dim))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn((n, heads, BT * dim), generator=gen, device="cuda").mul_(width)
        pool[i:i + n] = x.clamp_(-FMAX[fmt], FMAX[fmt]).to(F8[fmt]).view(torch.uint8)
    return pool


def _padded(scale):
    """The scale at the start of a buffer of whole 256-byte lines, as the pools keep it."""
    buf = torch.ones(-(-scale.numel() // 64) * 64, dtype=torch.float32, device="cuda")
    buf[: scale.numel()] = scale
    return buf[: scale.numel()]


def _kv_pools(blocks, heads, dim, fmt, per_head, gen):
    """A key pool (channels of very different sizes, two outliers a head) and a value pool, with their scales."""
    c = torch.exp(torch.randn((heads, dim), generator=gen, device="cuda"))
    c[:, :2] *= 10.0
    c = torch.gather(c, 1, torch.rand((heads, dim), generator=gen, device="cuda").argsort(1))
    top = c.amax(1) if per_head else c.amax().reshape(1)
    ks = 5.0 * top / FMAX[fmt]
    vs = 5.0 / FMAX[fmt] * (0.5 + torch.rand(heads if per_head else 1, generator=gen, device="cuda"))
    k = _random_pool(blocks, heads, dim, fmt, "k", c / (ks[:, None] if per_head else ks), gen)
    one = torch.ones((heads, dim), device="cuda")
    v = _random_pool(blocks, heads, dim, fmt, "v", one / (vs[:, None] if per_head else vs), gen)
    return k, v, _padded(ks), _padded(vs)


def _shared_tables(shared, extra, width, longest, blocks, cpu):
    """Block tables [groups * width, longest] of random distinct blocks: each group's rows begin with the same
    shared[g] of them, row b holds extra[b] more. Also the blocks left over."""
    perm = torch.randperm(blocks, generator=cpu)
    table = torch.full((extra.numel(), longest), -1)
    at = 0
    for g, n in enumerate(shared.tolist()):
        table[g * width:(g + 1) * width, :n] = perm[at:at + n]
        at += n
        for b in range(g * width, (g + 1) * width):
            m = int(extra[b])
            table[b, n:n + m] = perm[at:at + m]
            at += m
    return table.int(), perm[at:].int()


def _parents(groups, width, cpu):
    """A beam search's parents: of the beams sorted by score, the first ones survive more often and more than once."""
    x = (torch.rand((groups, width), generator=cpu) ** 2 * width).long().clamp_(max=width - 1)
    return x.sort(1).values


def prepare(case, seed):
    c = dict(case)
    cpu, gen = torch.Generator().manual_seed(seed), torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["op"] == "select":
        g, w, v = c["groups"], c["width"], c["vocab"]
        x = torch.empty((g * w, v), dtype=FLOAT[c["dtype"]], device="cuda")
        step = max(1, (1 << 27) // v)
        for i in range(0, g * w, step):
            # normal logits and, as a trained model's have, a few far above the rest
            y = torch.randn((min(step, g * w - i), v), generator=gen, device="cuda").mul_(2.0)
            y[:, : 40] += 6.0 + 3.0 * torch.randn((y.shape[0], 40), generator=gen, device="cuda")
            y = y.roll(int(torch.randint(v, (1,), generator=cpu)), 1)
            if c["banned"]:
                y.masked_fill_(torch.rand(y.shape, generator=gen, device="cuda") < c["banned"], -math.inf)
            x[i:i + step] = y.to(x.dtype)
        s["logits"] = x
        s["scores"] = (-30.0 - 5.0 * torch.rand((g, w), generator=gen, device="cuda")).sort(1, descending=True).values
        s["finished"] = torch.rand((g, w), generator=gen, device="cuda") < 0.2 if c["finished"] else None
        s["end_token"] = v // 3
    elif c["op"] == "fork":
        g, w = c["groups"], c["width"]
        shared = _spread(cpu, c["shared_lo"], c["shared_hi"], g)
        # the beams of a request are equally long
        tokens = shared.repeat_interleave(w) * BT + _spread(cpu, 1, c["own_hi"], g).repeat_interleave(w)
        held = -(-tokens // BT)
        extra = held - shared.repeat_interleave(w)
        blocks = int(shared.sum() + extra.sum()) + g * w + 5
        table, free = _shared_tables(shared, extra, w, c["shared_hi"] + -(-c["own_hi"] // BT) + 1, blocks, cpu)
        stack = torch.zeros(blocks, dtype=torch.int32)
        stack[: free.numel()] = free
        shares = torch.zeros(blocks, dtype=torch.int32)
        for i, n in enumerate(shared.tolist()):
            shares[table[i * w, :n].long()] = w - 1
        parents = _parents(g, w, cpu)
        if c["dropped"]:
            parents[torch.rand(g, generator=cpu) < 0.05] = -1
        s.update(table=table.cuda(), held=held.int().cuda(), lens=tokens.int().cuda(), parents=parents.int().view(-1).cuda(),
                 shares=shares.cuda(), free=stack.cuda(), free_count=torch.tensor([free.numel()], **i32),
                 src=torch.full((g * w,), -1, **i32), dst=torch.full((g * w,), -1, **i32), blocks=blocks)
    elif c["op"] == "copy":
        n = c["pairs"]
        size = c["block_bytes"]
        s["pools"] = [torch.randn((c["blocks"], size), generator=gen, device="cuda").to(F8["e4m3"]).view(torch.uint8)
                      for _ in range(c["buffers"])]
        perm = torch.randperm(c["blocks"], generator=cpu).int()
        s["src"], s["dst"] = perm[torch.randint(n, (n,), generator=cpu)].cuda(), perm[n:2 * n].cuda()
        s["count"] = torch.tensor([n], **i32)
    elif c["op"] == "compact":
        held = _spread(cpu, c["held_lo"], c["held_hi"], c["batch"])
        none = torch.zeros(c["batch"], dtype=torch.long)
        table, free = _shared_tables(none, held, 1, c["held_hi"], c["blocks"], cpu)
        stack = torch.zeros(c["blocks"], dtype=torch.int32)
        stack[: free.numel()] = free
        room = min(c["keep"], c["blocks"] - c["keep"])
        s.update(held=held.int().cuda(), src=torch.full((max(1, room),), -1, **i32), dst=torch.full((max(1, room),), -1, **i32))
        s["saved"] = [table.cuda(), torch.zeros(c["blocks"], **i32), stack.cuda(), torch.tensor([free.numel()], **i32)]
        s["work"] = [t.clone() for t in s["saved"]]
    else:
        g, w, h, hq, d = c["groups"], c["width"], c["heads"], c["q_heads"], c["dim"]
        shared = _spread(cpu, c["shared_lo"], c["shared_hi"], g)
        tail = _spread(cpu, c["own_lo"], c["own_hi"], g * w)
        extra = -(-tail // BT)
        blocks = int(shared.sum() + extra.sum()) + 3
        table, _ = _shared_tables(shared, extra, w, c["shared_hi"] + -(-c["own_hi"] // BT), blocks, cpu)
        kp, vp, ks, vs = _kv_pools(blocks, h, d, c["fmt"], c["per_head"], gen)
        q = torch.randn((g * w, hq, d), generator=gen, device="cuda", dtype=torch.float16)
        lens = shared.repeat_interleave(w) * BT + tail
        s.update(q=q, k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, table=table.cuda(), lens=lens.int().cuda(),
                 shared=shared.int().cuda(), longest=int(lens.max()), blocks=blocks)
    return s


# ---------------------------------------------------------------- plain forms

def _select_plain(s):
    c = s["case"]
    g, w, v, n = c["groups"], c["width"], c["vocab"], c["out"]
    # (64 bits: candidates of different beams may lie close to one another)
    x = s["logits"].double().view(g, w, v)
    x = x - x.amax(-1, keepdim=True)
    x = x - x.exp().sum(-1, keepdim=True).log() + s["scores"].double()[..., None]
    if s["finished"] is not None:
        x = torch.where(s["finished"][..., None], -math.inf, x)
        x[..., s["end_token"]] = torch.where(s["finished"], s["scores"].double(), x[..., s["end_token"]])
    x = x.view(g, w * v)
    # the n largest; among those equal to the last of them the lowest places
    top, at = x.topk(n, 1)
    last = top[:, -1:]
    places = torch.arange(w * v, device="cuda")
    equal = torch.where(x == last, w * v - places, 0).topk(n, 1).values
    at = torch.cat([torch.where(top > last, at, w * v), w * v - equal], 1).sort(1).values
    val = torch.where(at < w * v, x.gather(1, at.clamp(max=w * v - 1)), -math.inf)
    order = torch.sort(val, dim=1, descending=True, stable=True).indices[:, :n]
    at, val = at.gather(1, order), val.gather(1, order)
    return {"scores": val.float(), "parents": (at // v).int(), "tokens": (at % v).int()}


def _fork_plain(s):
    c = s["case"]
    g, w = c["groups"], c["width"]
    table, shares, stack, blocks = s["table"], s["shares"].long(), s["free"].long(), s["blocks"]
    b, width = table.shape
    col, row = torch.arange(width, device="cuda"), torch.arange(b, device="cuda")
    parent = s["parents"].long()
    alive = (parent >= 0) & (parent < w)
    source = row // w * w + torch.where(alive, parent, 0)
    lens = torch.where(alive, s["lens"].long()[source], 0)
    held = -(-lens // BT)
    old = torch.where(col < s["held"].long()[:, None], table.long(), -1)
    new = torch.where(col < held[:, None], old[source], -1)
    # references: a block that loses its last one is free; the lowest such block ends on top of the stack
    refs = torch.zeros(blocks + 1, dtype=torch.int64, device="cuda")
    refs.index_add_(0, torch.where(new >= 0, new, blocks).view(-1), torch.ones_like(new).view(-1))
    refs.index_add_(0, torch.where(old >= 0, old, blocks).view(-1), torch.full_like(old, -1).view(-1))
    shares = shares + refs[:blocks]
    freed = shares < 0
    shares = torch.where(freed, 0, shares)
    above = freed.sum() - torch.cumsum(freed, 0)
    stack = torch.cat([stack, stack.new_zeros(1)])
    stack = stack.scatter(0, torch.where(freed, s["free_count"].long() + above, blocks), torch.arange(blocks, device="cuda"))
    top = s["free_count"].long() + freed.sum()
    # a partly filled last block that several hold: the first beam keeps it where only such beams do, others copy
    partial = lens % BT != 0
    last = (held - 1).clamp(min=0)
    tail = torch.where(partial, new.gather(1, last[:, None])[:, 0], -1 - row)
    same = tail.view(g, w, 1) == tail.view(g, 1, w)
    first = ~(same & torch.ones((w, w), dtype=torch.bool, device="cuda").tril(-1)).any(-1).view(-1)
    among = same.sum(-1).view(-1)
    copier = partial & ~(first & (shares[tail.clamp(min=0)] + 1 == among))
    rank = torch.cumsum(copier, 0) - 1
    made = copier & (rank < top)
    fresh = stack[torch.where(made, top - 1 - rank, blocks)]
    shares = torch.cat([shares, shares.new_zeros(1)]).index_add(0, torch.where(made, tail, blocks), torch.full_like(tail, -1))[:blocks]
    new = new.scatter(1, last[:, None], torch.where(made, fresh, new.gather(1, last[:, None])[:, 0])[:, None])
    into = torch.where(made, rank, b)
    for name, val in (("src", tail), ("dst", fresh)):
        s[name] = torch.cat([s[name], s[name].new_zeros(1)]).scatter(0, into, val.int())[:b]
    # leading full blocks that the live beams of a request have in common
    live = (lens > 0).view(g, w)
    full = torch.where(live, (lens // BT).view(g, w), width).amin(1)
    t3 = new.view(g, w, width)
    lead = t3.gather(1, live.int().argmax(1).view(g, 1, 1).expand(g, 1, width))
    differ = ((t3 != lead) & live[..., None]).any(1)
    alike = torch.where(differ.any(1), differ.int().argmax(1), width)
    s["shared"] = torch.where(live.any(1), torch.minimum(full, alike), 0).int()
    s["table"], s["held"], s["lens"], s["shares"] = new.int(), held.int(), lens.int(), shares.int()
    s["free"], s["free_count"] = stack[:blocks].int(), (top - made.sum()).int()
    s["count"], s["granted"] = made.sum().int().view(1), (~copier | made).int()


def _compact_plain(s):
    c = s["case"]
    table, shares, stack, count = (t.long() for t in s["work"])
    blocks, keep, room = c["blocks"], c["keep"], s["src"].numel()
    place = torch.arange(blocks, device="cuda")
    free = torch.zeros(blocks + 1, dtype=torch.bool, device="cuda")
    free[torch.where(place < count, stack, blocks)] = True
    free = free[:blocks]
    mover, target = ~free & (place >= keep), free & (place < keep)
    n, t = mover.sum(), target.sum()
    done = (n <= t) & (n <= room)
    mover &= done
    m_rank, t_rank = torch.cumsum(mover, 0) - 1, torch.cumsum(target, 0) - 1
    targets = torch.zeros(blocks + 1, dtype=torch.int64, device="cuda").scatter(0, torch.where(target, t_rank, blocks), place)
    moved = torch.where(mover, targets[m_rank.clamp(min=0)], place)
    into = torch.where(mover, m_rank, room)
    src = torch.cat([s["src"], s["src"].new_zeros(1)]).scatter(0, into, place.int())[:room]
    dst = torch.cat([s["dst"], s["dst"].new_zeros(1)]).scatter(0, into, moved.int())[:room]
    held = torch.arange(table.shape[1], device="cuda") < s["held"][:, None]
    table = torch.where(held, moved[table.clamp(min=0)], table)
    shares = torch.where(mover, 0, shares).scatter_add(0, moved, torch.where(mover, shares, 0))
    left = target & (t_rank >= n) & done
    stack = torch.cat([stack, stack.new_zeros(1)]).scatter(0, torch.where(left, t - 1 - t_rank, blocks), place)[:blocks]
    for at, val in zip(s["work"], (table, shares, stack, torch.where(done, t - n, count))):
        at.copy_(val)
    return {"moved_to": moved.int(), "src": src, "dst": dst, "count": torch.where(done, n, 0).int().view(1),
            "done": done.int().view(1)}


def _values(pool, scale, blocks, dim, role, fmt):
    """Pool blocks [n, m] -> values [n, heads, m * 16, dim] in 32 bits."""
    n, m = blocks.shape
    h = pool.shape[1]
    order = _order(dim, role).view(-1)
    x = pool[blocks.clamp(min=0)].view(F8[fmt])                       # [n, m, heads, 16 * dim]
    x = x.view(torch.uint8)[..., order].view(F8[fmt]).float().view(n, m, h, BT, dim)
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, m * BT, dim) * scale.view(1, -1, 1, 1)


def _attend_plain(s):
    c = s["case"]
    g, w, h, d = c["groups"], c["width"], c["heads"], c["dim"]
    gq = c["q_heads"] // h
    table, lens, shared = s["table"].long(), s["lens"].long(), s["shared"].long()
    q = s["q"].float().view(g, w, h, gq, d)
    p, e = c["shared_hi"], -(-c["own_hi"] // BT)
    scale = 1.0 / math.sqrt(d)
    parts = []                                                        # (scores, values) of the shared and of the own tokens
    if p > 0:
        blocks = table.view(g, w, -1)[:, 0, :p]
        k = _values(s["k_pool"], s["k_scale"], blocks, d, "k", c["fmt"])
        x = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(g, h, w * gq, d), k.transpose(2, 3)).view(g, h, w, gq, -1) * scale
        del k
        x.masked_fill_((torch.arange(p * BT, device="cuda") >= shared[:, None] * BT).view(g, 1, 1, 1, -1), -math.inf)
        parts.append(x)
    first = shared.repeat_interleave(w)[:, None]
    at = (first + torch.arange(e, device="cuda")).clamp(max=table.shape[1] - 1)
    tail = table.gather(1, at)
    seen = torch.arange(e * BT, device="cuda") < (lens[:, None] - first * BT)
    k = _values(s["k_pool"], s["k_scale"], tail, d, "k", c["fmt"])     # [g * w, h, e * 16, d]
    x = torch.matmul(q.view(g * w, h, gq, d), k.transpose(2, 3)) * scale
    del k
    x.masked_fill_(~seen[:, None, None, :], -math.inf)
    parts.append(x.view(g, w, h, gq, -1).permute(0, 2, 1, 3, 4))
    top = parts[0].amax(-1, keepdim=True)
    for x in parts[1:]:
        top = torch.maximum(top, x.amax(-1, keepdim=True))
    parts = [(x - top).exp_() for x in parts]
    total = sum(x.sum(-1, keepdim=True) for x in parts)
    v = _values(s["v_pool"], s["v_scale"], tail, d, "v", c["fmt"])
    v = torch.where(seen[:, None, :, None], v, 0.0)
    o = torch.matmul(parts[-1].permute(0, 2, 1, 3, 4).reshape(g * w, h, gq, -1), v).view(g, w, h, gq, d)
    del v
    if p > 0:
        v = _values(s["v_pool"], s["v_scale"], blocks, d, "v", c["fmt"])
        o = o + torch.matmul(parts[0].reshape(g, h, w * gq, -1), v).view(g, h, w, gq, d).permute(0, 2, 1, 3, 4)
    return (o / total.permute(0, 2, 1, 3, 4)).half().view(g * w, h * gq, d)


# ---------------------------------------------------------------- a pass

def _handles(s):
    """The descriptors, workspaces and result buffers that a user's program keeps."""
    if "handles" in s:
        return s["handles"]
    from quantized_kv_cache_quant_gb300 import beam, kvq
    c = s["case"]
    i32 = dict(dtype=torch.int32, device="cuda")
    if c["op"] == "select":
        shape = (c["groups"], c["out"])
        made = [torch.empty(shape, dtype=torch.float32, device="cuda"), torch.empty(shape, **i32), torch.empty(shape, **i32)]
    elif c["op"] == "fork":
        s.update(count=torch.zeros(1, **i32), granted=torch.empty(c["groups"] * c["width"], **i32),
                 shared=torch.empty(c["groups"], **i32))
        made = [beam.blocks_workspace(c["groups"], s["blocks"])]
    elif c["op"] == "copy":
        made = [beam.BlockBuffers(c["blocks"], s["pools"])]
    elif c["op"] == "compact":
        made = [torch.empty(c["blocks"], **i32), torch.zeros(1, **i32), torch.zeros(1, **i32),
                beam.blocks_workspace(1, c["blocks"])]
    else:
        fmt = kvq.FP8_FORMATS[c["fmt"]]
        made = [kvq.fp8_pool_init(role, fmt, c["per_head"], s["blocks"], c["heads"], c["dim"], pool, scale)
                for role, pool, scale in ((kvq.ROLE_KEY, s["k_pool"], s["k_scale"]), (kvq.ROLE_VALUE, s["v_pool"], s["v_scale"]))]
        made.append(beam.group_workspace(c["groups"] * c["width"], c["heads"], c["q_heads"], c["dim"], c["width"]))
    s["handles"] = made
    return made


def run(s):
    c = s["case"]
    if own:
        from quantized_kv_cache_quant_gb300 import beam
    if c["op"] == "select":
        if not own:
            return _select_plain(s)
        scores, parents, tokens = _handles(s)
        beam.beam_select(s["logits"], s["scores"], scores, parents, tokens, s["finished"], s["end_token"])
        return {"scores": scores, "parents": parents, "tokens": tokens}
    if c["op"] == "fork":
        # the parents are the same in every pass: copies are made and replaced ones come back in each of them
        if own:
            (ws,) = _handles(s)
            beam.kv_blocks_fork(s["table"], s["held"], s["lens"], s["parents"], c["width"], BT, s["shares"], s["free"],
                                s["free_count"], s["src"], s["dst"], s["count"], ws, s["granted"], s["shared"])
        else:
            _fork_plain(s)
        return {name: s[name] for name in ("table", "held", "lens", "shares", "free", "free_count", "src", "dst", "count",
                                           "granted", "shared")}
    if c["op"] == "copy":
        if own:
            beam.kv_blocks_copy(_handles(s)[0], s["src"], s["dst"], s["count"])
        else:
            for pool in s["pools"]:
                pool[s["dst"].long()] = pool[s["src"].long()]
        return [pool.view(F8["e4m3"]) for pool in s["pools"]]
    if c["op"] == "compact":
        # the tables of before the pass: a second pass over a compact pool would have nothing to do
        torch._foreach_copy_(s["work"], s["saved"])
        table, shares, stack, count = s["work"]
        if own:
            moved, n, done, ws = _handles(s)
            beam.kv_blocks_compact(table, s["held"], c["keep"], shares, stack, count, moved, s["src"], s["dst"], n, done, ws)
            out = {"moved_to": moved, "src": s["src"], "dst": s["dst"], "count": n, "done": done}
        else:
            out = _compact_plain(s)
        return dict(out, table=table, shares=shares, free=stack, free_count=count)
    if not own:
        return _attend_plain(s)
    k, v, ws = _handles(s)
    out = torch.empty(s["q"].shape, dtype=torch.float16, device="cuda")
    beam.fp8_group_attention(s["q"], k, v, s["table"], s["lens"], s["shared"], c["width"], s["longest"], out, 0.0, ws)
    return out


# ---------------------------------------------------------------- floors

def work(case):
    c = case
    if c["op"] == "select":
        rows = c["groups"] * c["width"]
        size = 4.0 if c["dtype"] == "fp32" else 2.0
        # every logit once (a beam that has ended needs none: a fifth of them), an exponential's few operations each
        live = 0.8 if c["finished"] else 1.0
        return {"bytes": live * rows * c["vocab"] * size + 4.0 * rows + 12.0 * c["groups"] * c["out"],
                "flops": 4.0 * live * rows * c["vocab"]}
    if c["op"] == "fork":
        rows = c["groups"] * c["width"]
        blocks = (c["shared_lo"] + c["shared_hi"]) / 2 + c["own_hi"] / 2 / BT
        # every table entry read once; what changes (a few blocks a beam) written, with counts and copies
        return {"bytes": rows * (4.0 * blocks + 100.0), "flops": 0}
    if c["op"] == "copy":
        return {"bytes": c["buffers"] * c["pairs"] * 2.0 * c["block_bytes"], "flops": 0}
    if c["op"] == "compact":
        entries = c["batch"] * (c["held_lo"] + c["held_hi"]) / 2
        moved = entries * (1.0 - c["keep"] / c["blocks"])
        # the free blocks read, the new places, every table entry read, and what moves written: entry, pair, counts
        return {"bytes": 4.0 * (c["blocks"] - entries) + 4.0 * c["blocks"] + 4.0 * entries + 20.0 * moved
                + 4.0 * (c["keep"] - entries), "flops": 0}
    rows, d = c["groups"] * c["width"], c["dim"]
    shared, tail = BT * (c["shared_lo"] + c["shared_hi"]) / 2, (c["own_lo"] + c["own_hi"]) / 2
    return {"bytes": 2.0 * c["heads"] * d * (c["groups"] * shared + rows * tail) + 4.0 * rows * c["q_heads"] * d,
            "flops": 4.0 * rows * c["q_heads"] * (shared + tail) * d}


# ---------------------------------------------------------------- from the definitions, in 64 bits

def _code_values(fmt):
    """The 256 codes' values by their bit fields, in 64 bits."""
    bits, bias = (3, 7) if fmt == "e4m3" else (2, 15)
    v = []
    for code in range(256):
        e, m = code >> bits & (1 << (7 - bits)) - 1, code & (1 << bits) - 1
        x = math.ldexp(m, 1 - bias - bits) if e == 0 else math.ldexp((1 << bits) + m, e - bias - bits)
        if code & 0x7F == 0x7F or fmt == "e5m2" and e == 31 and m:
            x = math.nan
        elif fmt == "e5m2" and e == 31:
            x = math.inf
        v.append(-x if code >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def exact(case, seed):
    if case["op"] in ("fork", "copy", "compact"):
        return None                                   # whole numbers and moved bytes: compared with the plain form's
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "select":
        out = torch.empty((c["groups"], c["out"]), dtype=torch.float64, device="cuda")
        for g in range(c["groups"]):
            rows = []
            for b in range(c["width"]):
                score = s["scores"][g, b].double()
                if s["finished"] is not None and bool(s["finished"][g, b]):
                    rows.append(score.view(1))
                    continue
                x = s["logits"][g * c["width"] + b].double()
                rows.append((x - torch.logsumexp(x, 0) + score).sort(descending=True).values[: c["out"]])
            best = torch.cat(rows).sort(descending=True).values[: c["out"]]
            out[g, : best.numel()] = best
            out[g, best.numel():] = -math.inf
        return {"scores": out, "parents": None, "tokens": None}
    d, gq, w = c["dim"], c["q_heads"] // c["heads"], c["width"]
    val = _code_values(c["fmt"])
    offs = {"k": _order(d, "k").reshape(-1), "v": _order(d, "v").reshape(-1)}
    lens, table = s["lens"].tolist(), s["table"].long()
    rows = c["groups"] * w
    if rows * c["heads"] * max(lens) * d * (2 + gq) > 3e11:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(rows):
        n = lens[b]
        blocks = table[b, : -(-n // BT)]
        for h in range(c["heads"]):
            kv = {}
            for name in ("k", "v"):
                raw = s[name + "_pool"][blocks, h][:, offs[name]].reshape(-1, d)[:n]
                scale = s[name + "_scale"]
                kv[name] = val[raw.long()] * scale.double()[h if scale.numel() > 1 else 0]
            x = s["q"][b, h * gq:(h + 1) * gq].double() @ kv["k"].T / math.sqrt(d)
            p = torch.softmax(x, 1)
            out[b, h * gq:(h + 1) * gq] = p @ kv["v"]
    return out
