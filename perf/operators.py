"""Performance cases of the speculative-decoding operators over the paged FP8 cache.

One step of a serving loop that verifies drafted tokens: the block tables grow,
the new tokens' slots are mapped, keys and values are appended in FP8, a tree
of drafted tokens attends over the cache, the accepted path moves to the front.
Each case is one of these operators at a size such a loop meets. `run` computes
it in elementary torch operations, or with `own` through the library.
"""
import math

import torch

own = False

BT = 16                      # tokens of a pool block
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ---------------------------------------------------------------- cases

def _plan(name, batch, ctx_lo, ctx_hi, new_lo, new_hi, max_blocks):
    return {"name": name, "op": "plan", "batch": batch, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "new_lo": new_lo,
            "new_hi": new_hi, "max_blocks": max_blocks}


def _append(name, tokens, run, heads, dim, fmt, per_head, fused, q_heads):
    """`run`: tokens a request appends one after the other (their slots are neighbours)."""
    return {"name": name, "op": "append", "tokens": tokens, "run": run, "heads": heads, "dim": dim, "fmt": fmt,
            "per_head": per_head, "fused": fused, "q_heads": q_heads}


def _accept(name, batch, heads, dim, ctx_lo, ctx_hi, tree, path):
    return {"name": name, "op": "accept", "batch": batch, "heads": heads, "dim": dim, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "tree": tree, "path": path}


def _attend(name, batch, heads, q_heads, dim, ctx_lo, ctx_hi, tree_lo, tree_hi, fmt="e4m3", per_head=False,
            fused=False):
    return {"name": name, "op": "attend", "batch": batch, "heads": heads, "q_heads": q_heads, "dim": dim,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "tree_lo": tree_lo, "tree_hi": tree_hi, "fmt": fmt,
            "per_head": per_head, "fused": fused}


def listed():
    return [
        # a small server's step: each of 8 requests adds a handful of drafted tokens
        _plan("plan_step_b8", 8, 100, 4000, 1, 8, 512),
        # admission of 256 prompts of up to 16K tokens at once, and their release
        _plan("plan_admit_b256", 256, 0, 0, 512, 16384, 1024),
        # one drafted token for each of 8 requests, latency bound
        _append("append_8", 8, 1, 8, 128, "e4m3", False, False, 32),
        # 64 requests with trees of 33 nodes, keys and values taken from a fused projection's rows
        _append("append_trees_2112", 2112, 33, 8, 64, "e5m2", True, True, 16),
        # a long prompt chunk
        _append("append_chunk_65536", 65536, 8192, 8, 128, "e4m3", False, True, 32),
        # one request's accepted path
        _accept("accept_b1", 1, 8, 128, 1000, 1000, 16, 4),
        # a full server's accepted paths
        _accept("accept_b256", 256, 8, 128, 200, 1500, 60, 12),
        # one request with a short chain, latency bound
        _attend("tree_b1_s1000_t5", 1, 8, 32, 128, 1000, 1000, 5, 5),
        # chains of 4 over the 128K streaming cache, 8 query heads per kv head: 32 rows a kv head, few requests
        _attend("tree_b4_s131072_t4", 4, 8, 64, 128, 131072, 131072, 4, 4),
        # the 32K serving cache with trees of 16: 64 rows a kv head
        _attend("tree_b32_s32768_t16", 32, 8, 32, 128, 32768, 32768, 16, 16, fused=True),
        # large trees: 8 query heads x 63 nodes = 504 rows a kv head, bound by the products
        _attend("tree_b16_s16384_t63", 16, 8, 64, 128, 16384, 16384, 63, 63),
        # ragged lengths and trees, 64 channels, E5M2 with a scale per head
        _attend("tree_b32_ragged", 32, 8, 32, 64, 512, 16384, 1, 40, "e5m2", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "accept", "attend", "attend", "attend"])
    heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    fmt, per_head, fused = rng.choice(["e4m3", "e5m2"]), rng.random() < 0.5, rng.random() < 0.5
    if op == "plan":
        batch = _log(rng, 1, 256)
        lo, new = _log(rng, 1, 4000), _log(rng, 1, 12000)
        hi = lo + _log(rng, 1, 3000)
        c = _plan("", batch, lo, hi, max(0, new // _log(rng, 1, 20) - 1), new, (hi + new) // BT + 1 + rng.randrange(20))
    elif op == "append":
        run = _log(rng, 1, 400)
        c = _append("", _log(rng, 1, 40000), run, heads, dim, fmt, per_head, fused, heads * rng.choice([1, 2, 4, 8]))
    elif op == "accept":
        tree = _log(rng, 1, 64)
        lo = rng.randrange(0, 1500)
        c = _accept("", _log(rng, 1, 256), heads, dim, lo, lo + rng.randrange(500), tree, rng.randint(1, min(tree, 16)))
    else:
        tree = _log(rng, 1, 128)
        gq = rng.choice([1, 2, 4, 8])
        lo = _log(rng, 1, 100000) - 1
        hi = lo + _log(rng, 1, 8000)
        # at most about as many query rows x context tokens as the largest listed case
        most = 16 * 8 * 504 * 16384 // (heads * gq * tree * (hi + 1))
        c = _attend("", max(1, min(_log(rng, 1, 64), most, 2_000_000 // (hi + 1))), heads, heads * gq, dim, lo, hi,
                    max(1, tree // rng.choice([1, 2, 8])), tree, fmt, per_head, fused)
    del c["name"]
    return c


# ---------------------------------------------------------------- inputs

def _spread(gen, lo, hi, n):
    """n whole numbers spread evenly over lo .. hi, in a random order: their sum goes by the case alone."""
    x = torch.arange(n) * (hi - lo) // max(1, n - 1) + lo if n > 1 else torch.tensor([hi])
    return x[torch.randperm(n, generator=gen)]


def _to_f8(y, fmt):
    m = FMAX[fmt]
    return y.clamp_(-m, m).to(F8[fmt])


def _fill_pool(blocks, heads, dim, fmt, gen, spread):
    """Random pool bytes [blocks, heads, 16 * dim] whose channels differ in size, as keys' do. The places of a
    block's bytes are drawn alike for all its tokens, so the order within the block does not matter here: every
    channel keeps its size through _offsets."""
    pool = torch.empty((blocks, heads, BT * dim), dtype=torch.uint8, device="cuda")
    role, width = spread
    off = _offsets(dim, role).reshape(-1)
    size = torch.empty((heads, BT * dim), device="cuda")
    size[:, off] = width.repeat(1, BT)
    step = max(1, (1 << 26) // (heads * BT * dim))
    for i in range(0, blocks, step):
        n = min(step, blocks - i)
        x = torch.randn((n, heads, BT * dim), generator=gen, device="cuda", dtype=torch.float32).mul_(size)
        pool[i:i + n] = _to_f8(x, fmt).view(torch.uint8)
    return pool


def _pools(blocks, heads, dim, fmt, per_head, gen):
    """A key pool (channels of very different sizes, two outliers a head) and a value pool, with their scales: the
    scale takes 5 standard deviations of the largest channel to the format's maximum."""
    c = torch.exp(torch.randn((heads, dim), generator=gen, device="cuda"))
    c[:, :2] *= 10.0
    c = torch.gather(c, 1, torch.rand((heads, dim), generator=gen, device="cuda").argsort(1))
    top = c.amax(1) if per_head else c.amax().reshape(1)
    m = FMAX[fmt]
    k_scale = (5.0 * top / m).float().contiguous()
    k_pool = _fill_pool(blocks, heads, dim, fmt, gen, ("k", c / (k_scale[:, None] if per_head else k_scale)))
    n = heads if per_head else 1
    v_scale = (5.0 / m * (0.5 + torch.rand(n, generator=gen, device="cuda"))).contiguous()
    width = torch.ones((heads, dim), device="cuda") / (v_scale[:, None] if per_head else v_scale)
    v_pool = _fill_pool(blocks, heads, dim, fmt, gen, ("v", width))
    return k_pool, v_pool, _slot256(k_scale), _slot256(v_scale)


def _slot256(scale):
    """The scale at the start of a buffer of whole 256-byte lines, as the pools keep it."""
    buf = torch.ones(-(-scale.numel() // 64) * 64, dtype=torch.float32, device="cuda")
    buf[: scale.numel()] = scale
    return buf[: scale.numel()]


def _offsets(dim, role, device="cuda"):
    """Byte of (token row, channel) in a block of 16 x dim: int64 [16, dim]."""
    t, c = torch.arange(BT, device=device)[:, None], torch.arange(dim, device=device)[None, :]
    if role == "k":
        chunk, lane, byte = (t // 8) * (dim // 64) + c // 64, 4 * (t % 8) + c % 16 // 4, c % 64 // 16 * 4 + c % 4
    else:
        chunk, lane, byte = c // 32, 4 * (c % 8) + t % 8 // 2, c % 32 // 8 * 4 + t // 8 * 2 + t % 2
    return (chunk * 32 + lane) * 16 + byte


def _tables(held, max_blocks, num_blocks, cpu):
    """Distinct random blocks for each request's `held` entries (-1 behind), and the blocks left over."""
    perm = torch.randperm(num_blocks, generator=cpu)
    start = torch.cumsum(held, 0) - held
    j = torch.arange(max_blocks)[None, :]
    at = (start[:, None] + j).clamp_(max=num_blocks - 1)
    table = torch.where(j < held[:, None], perm[at], torch.tensor(-1))
    return table.to(torch.int32), perm[int(held.sum()):].to(torch.int32)


def _trees(lens, words, cpu):
    """Ancestor masks of random trees, node by node: int64 words [sum(lens), words]."""
    rows = []
    for n in lens.tolist():
        up = torch.randint(1, 7, (n,), generator=cpu).tolist()
        seen = []
        for i in range(n):
            p = i - up[i]
            seen.append((seen[p] if p >= 0 else 0) | (1 << i))
        rows += seen
    sign = lambda w: w - (1 << 64) if w >> 63 else w  # noqa: E731
    return torch.tensor([[sign(r >> (64 * w) & (1 << 64) - 1) for w in range(words)] for r in rows], dtype=torch.int64)


def prepare(case, seed):
    c = dict(case)
    cpu, gen = torch.Generator().manual_seed(seed), torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": c}
    if c["op"] == "plan":
        b = c["batch"]
        ctx, new = _spread(cpu, c["ctx_lo"], c["ctx_hi"], b), _spread(cpu, c["new_lo"], c["new_hi"], b)
        held = -(-ctx // BT)
        blocks = int((-(-ctx // BT) - -new // BT).sum()) + 7
        table, free = _tables(held, c["max_blocks"], blocks, cpu)
        stack = torch.zeros(blocks, dtype=torch.int32)
        stack[: free.numel()] = free
        s.update(table=table, held=held.int(), seq_lens=ctx.int(), new_lens=new.int(), grown=(ctx + new).int(),
                 free=stack, free_count=torch.tensor([free.numel()], dtype=torch.int32))
        s = {k: v.cuda() if torch.is_tensor(v) else v for k, v in s.items()}
        n = int(new.sum())
        s.update(num_blocks=blocks, rows=max(1, n + 3))
    elif c["op"] == "append":
        n, run, h, d = c["tokens"], c["run"], c["heads"], c["dim"]
        per = -(-(run + 1) // BT) + 1
        reqs = -(-n // run)
        blocks = reqs * per
        perm = torch.randperm(blocks, generator=cpu).view(reqs, per)
        i = torch.arange(n)
        pos = _spread(cpu, 0, BT - 1, reqs)[i // run] + i % run
        s["slots"] = (perm[i // run, pos // BT] * BT + pos % BT).cuda()
        kp, vp, ks, vs = _pools(blocks, h, d, c["fmt"], c["per_head"], gen)
        rows = (c["q_heads"] + 2 * h) * d if c["fused"] else h * d
        both = [torch.randn((n, rows), generator=gen, device="cuda", dtype=torch.float16) for _ in range(1 if c["fused"] else 2)]
        at = c["q_heads"] * d
        s["k_new"] = (both[0][:, at:at + h * d] if c["fused"] else both[0]).unflatten(1, (h, d))
        s["v_new"] = (both[0][:, at + h * d:] if c["fused"] else both[1]).unflatten(1, (h, d))
        s.update(k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, num_blocks=blocks)
    elif c["op"] == "accept":
        b = c["batch"]
        lens = _spread(cpu, c["ctx_lo"], c["ctx_hi"], b)
        held = -(-(lens + c["tree"]) // BT)
        blocks = int(held.sum()) + 3
        table, _ = _tables(held, int(held.max()), blocks - 1, cpu)      # the last block pads
        kp, vp, ks, vs = _pools(blocks, c["heads"], c["dim"], "e4m3", False, gen)
        path = torch.rand((b, c["tree"]), generator=cpu).argsort(1)[:, :c["path"]].sort(1).values
        s.update(k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, table=table.cuda(), seq_lens=lens.int().cuda(),
                 path=path.int().cuda(), accepted=_spread(cpu, 0 if b > 1 else c["path"], c["path"], b).int().cuda(), num_blocks=blocks)
    else:
        b, h, hq, d = c["batch"], c["heads"], c["q_heads"], c["dim"]
        lens, trees = _spread(cpu, c["ctx_lo"], c["ctx_hi"], b), _spread(cpu, c["tree_lo"], c["tree_hi"], b)
        held = -(-(lens + trees) // BT)
        blocks = int(held.sum()) + 3
        table, _ = _tables(held, int(held.max()), blocks, cpu)
        kp, vp, ks, vs = _pools(blocks, h, d, c["fmt"], c["per_head"], gen)
        n = int(trees.sum())
        wide = (hq + 2 * h) * d if c["fused"] else hq * d
        q = torch.randn((n, wide), generator=gen, device="cuda", dtype=torch.float16)[:, :hq * d].unflatten(1, (hq, d))
        offsets = torch.zeros(b + 1, dtype=torch.int32)
        offsets[1:] = torch.cumsum(trees, 0)
        s.update(k_pool=kp, v_pool=vp, k_scale=ks, v_scale=vs, table=table.cuda(), seq_lens=lens.int().cuda(), q=q,
                 offsets=offsets.cuda(), mask=_trees(trees, -(-c["tree_hi"] // 64), cpu).cuda(),
                 max_tree=int(trees.max()), max_seq=int((lens + trees).max()), num_blocks=blocks)
    return s


# ---------------------------------------------------------------- plain forms

def _resize(table, held, target, free, count):
    """The block tables after every request holds what `target` tokens need: (table, held, free, count, granted)."""
    b, width = table.shape
    blocks = free.numel()
    need = (target.long() + BT - 1) // BT
    ok = (target >= 0) & (need <= width)
    need = torch.where(ok, need, held.long())
    grow, drop = (need - held).clamp(min=0), (held - need).clamp(min=0)
    j = torch.arange(width, device=table.device)[None, :]
    f, r = count.long(), drop.sum()
    # released blocks, first one on top
    out = (j >= need[:, None]) & (j < held[:, None])
    rank = (torch.cumsum(drop, 0) - drop)[:, None] + j - need[:, None]
    stack = torch.cat([free, free.new_zeros(1)])
    stack = stack.scatter(0, torch.where(out, f + r - 1 - rank, blocks).reshape(-1), table.reshape(-1))
    table = torch.where(out, -1, table)
    # new blocks from the top, in the order of the requests, while they last
    granted = ok & ((grow == 0) | (torch.cumsum(grow, 0) <= f + r))
    grow = torch.where(granted, grow, 0)
    rank = (torch.cumsum(grow, 0) - grow)[:, None] + j - held[:, None]
    into = (j >= held[:, None]) & (j < (held + grow)[:, None])
    table = torch.where(into, stack[torch.where(into, f + r - 1 - rank, blocks)], table)
    held = torch.where(granted, need, held.long())
    return table, held.int(), stack[:blocks], (f + r - grow.sum()).int(), granted.int()


def _slots(table, seq_lens, new_lens, blocks, rows):
    """Slot, request and position of each new token, and the requests' offsets."""
    b, width = table.shape
    offsets = torch.nn.functional.pad(torch.cumsum(new_lens, 0), (1, 0)).int()
    i = torch.arange(rows, device=table.device)
    seq = torch.searchsorted(offsets[1:].long(), i, right=True)
    live = seq < b
    seq = seq.clamp(max=b - 1)
    pos = seq_lens[seq].long() + i - offsets[seq]
    block = table[seq, (pos // BT).clamp(max=width - 1)].long()
    good = live & (pos < width * BT) & (block >= 0) & (block < blocks)
    slots = torch.where(good, block * BT + pos % BT, -1)
    return offsets, slots, torch.where(live, seq, -1).int(), torch.where(live, pos, -1).int()


def _natural(blocks, dim, role, fmt):
    """Pool blocks [..., 16 * dim] bytes -> values [..., 16, dim] in 32 bits."""
    lead = blocks.shape[:-1]
    n = len(lead)
    if role == "k":      # token (2, 8), channel (64s, 16s, 4s, 1s)
        x = blocks.view(*lead, 2, dim // 64, 8, 4, 4, 4).permute(*range(n), n, n + 2, n + 1, n + 4, n + 3, n + 5)
    else:                # token (8s, 2s, 1s), channel (32s, 8s, 1s)
        x = blocks.view(*lead, dim // 32, 8, 4, 4, 2, 2).permute(*range(n), n + 4, n + 2, n + 5, n, n + 3, n + 1)
    return x.reshape(*lead, BT, dim).view(F8[fmt]).float()


def _write(pool, x, scale, slots, role, fmt):
    y = x.float() / (scale[:, None] if scale.numel() > 1 else scale)
    byte = _to_f8(y, fmt).view(torch.uint8)
    n, h, d = x.shape
    off = _offsets(d, role)[slots % BT]                                        # [n, d]
    at = ((slots // BT)[:, None] * h + torch.arange(h, device=pool.device))[:, :, None] * (BT * d) + off[:, None, :]
    pool.view(-1)[at.reshape(-1)] = byte.reshape(-1)


def _move_rows(pool, dim, role, table, src, dst, moved):
    """Each request's tokens at positions `src` to `dst` where `moved`."""
    blocks, h = pool.shape[:2]
    off = _offsets(dim, role)
    b = torch.arange(table.shape[0], device=pool.device)[:, None]
    heads = torch.arange(h, device=pool.device)[:, None]

    def places(pos):
        # what does not move stays within the pool's last block, which no table names
        block = torch.where(moved, table[b, (pos // BT).clamp(max=table.shape[1] - 1)].long(), blocks - 1)
        return (block[:, :, None, None] * h + heads) * (BT * dim) + off[torch.where(moved, pos % BT, 0)][:, :, None, :]

    flat = pool.view(-1)
    flat[places(dst)] = flat[places(src)]


def _attention(s):
    c = s["case"]
    table, lens, dim, fmt = s["table"].long(), s["seq_lens"].long(), c["dim"], c["fmt"]
    b, h, gq = table.shape[0], c["heads"], c["q_heads"] // c["heads"]
    n, t = s["q"].shape[0], s["max_tree"]
    first, count = s["offsets"][:-1].long(), (s["offsets"][1:] - s["offsets"][:-1]).long()
    # queries of each request, padded to the largest tree: [b, h, t * gq, dim]
    node = torch.arange(t, device="cuda")
    row = (first[:, None] + node).clamp(max=n - 1)
    q = s["q"].float()[row].view(b, t, h, gq, dim).permute(0, 2, 1, 3, 4).reshape(b, h, t * gq, dim)
    # what each node sees: [b, t, tokens]
    pos = torch.arange(table.shape[1] * BT, device="cuda")
    j = pos[None, :] - lens[:, None]
    inside = (j >= 0) & (j < count[:, None])
    jj = j.clamp(0, s["mask"].shape[1] * 64 - 1)
    word = torch.gather(s["mask"][row], 2, (jj // 64)[:, None, :].expand(b, t, -1))
    sees = (j < 0)[:, None, :] | (inside[:, None, :] & ((word >> (jj % 64)[:, None, :]) & 1).bool())
    used = (j < count[:, None])[:, None, :, None]
    at = table.clamp(min=0)

    def values(pool, role, scale):
        x = _natural(pool[at], dim, role, fmt).permute(0, 2, 1, 3, 4).reshape(b, h, -1, dim)
        x *= scale.view(1, -1, 1, 1)
        return torch.where(used, x, 0.0)

    scores = torch.matmul(q, values(s["k_pool"], "k", s["k_scale"]).transpose(2, 3)) * (1.0 / math.sqrt(dim))
    scores = scores.view(b, h, t, gq, -1).masked_fill_(~sees[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_(min=-3.0e38)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, h, t * gq, -1), values(s["v_pool"], "v", s["v_scale"])).view(b, h, t, gq, dim)
    o = (o / torch.where(total > 0, total, 1.0)).half().permute(0, 2, 1, 3, 4).reshape(b, t, h * gq, dim)
    owner = torch.searchsorted(s["offsets"][1:].long(), torch.arange(n, device="cuda"), right=True)
    return o[owner, torch.arange(n, device="cuda") - first[owner]]


# ---------------------------------------------------------------- a pass

def _handles(s):
    """The descriptors, the workspace and the index buffers that a user's program keeps beside its pools."""
    if "handles" not in s:
        from quantized_kv_cache_quant_gb300 import kvq, spec
        c = s["case"]
        if c["op"] == "plan":
            i32 = dict(dtype=torch.int32, device=s["table"].device)
            s["handles"] = [torch.empty(c["batch"], **i32), torch.empty(c["batch"] + 1, **i32),
                            torch.empty(s["rows"], dtype=torch.int64, device=s["table"].device),
                            torch.empty(s["rows"], **i32), torch.empty(s["rows"], **i32)]
            return s["handles"]
        fmt, ph = kvq.FP8_FORMATS[c.get("fmt", "e4m3")], c.get("per_head", False)
        made = [kvq.fp8_pool_init(role, fmt, ph, s["num_blocks"], c["heads"], c["dim"], pool, scale)
                for role, pool, scale in ((kvq.ROLE_KEY, s["k_pool"], s["k_scale"]), (kvq.ROLE_VALUE, s["v_pool"], s["v_scale"]))]
        if c["op"] == "attend":
            size = spec.fp8_tree_workspace_bytes(c["batch"], c["heads"], c["q_heads"], c["dim"], s["max_tree"])
            made.append(torch.zeros(size, dtype=torch.uint8, device="cuda"))
        s["handles"] = made
    return s["handles"]


def _plan_own(s):
    from quantized_kv_cache_quant_gb300 import spec
    granted, offsets, slots, seq, pos = _handles(s)
    spec.kv_blocks_resize(s["table"], s["held"], s["grown"], BT, s["free"], s["free_count"], granted)
    spec.kv_slot_map(s["table"], s["seq_lens"], s["new_lens"], BT, s["num_blocks"], offsets, slots, seq, pos)
    spec.kv_blocks_resize(s["table"], s["held"], s["seq_lens"], BT, s["free"], s["free_count"])
    return granted, offsets, slots, seq, pos


def run(s):
    c = s["case"]
    if c["op"] == "plan":
        # grow, map, and give the blocks back: the tables end as they began, so every pass does the same work
        if own:
            granted, offsets, slots, seq, pos = _plan_own(s)
        else:
            table, held, free, count, granted = _resize(s["table"], s["held"], s["grown"], s["free"], s["free_count"])
            offsets, slots, seq, pos = _slots(table, s["seq_lens"], s["new_lens"], s["num_blocks"], s["rows"])
            table, held, free, count, _ = _resize(table, held, s["seq_lens"], free, count)
            s["table"], s["held"], s["free"], s["free_count"] = table, held, free, count
        return {"granted": granted, "offsets": offsets, "slots": slots, "seq": seq, "pos": pos, "table": s["table"],
                "held": s["held"], "free": s["free"], "free_count": s["free_count"]}
    if c["op"] == "append":
        if own:
            from quantized_kv_cache_quant_gb300 import spec
            k, v = _handles(s)
            spec.fp8_kv_append(k, v, s["k_new"], s["v_new"], s["slots"])
        else:
            _write(s["k_pool"], s["k_new"], s["k_scale"], s["slots"], "k", c["fmt"])
            _write(s["v_pool"], s["v_new"], s["v_scale"], s["slots"], "v", c["fmt"])
        return {"k": s["k_pool"].view(F8[c["fmt"]]), "v": s["v_pool"].view(F8[c["fmt"]])}
    if c["op"] == "accept":
        new = torch.empty_like(s["seq_lens"])
        if own:
            from quantized_kv_cache_quant_gb300 import spec
            k, v = _handles(s)
            spec.fp8_kv_accept(k, v, s["table"], s["seq_lens"], s["path"], s["accepted"], new)
        else:
            i = torch.arange(c["path"], device="cuda")[None, :]
            src, dst = s["seq_lens"][:, None].long() + s["path"], s["seq_lens"][:, None].long() + i
            moved = i < s["accepted"][:, None]
            _move_rows(s["k_pool"], c["dim"], "k", s["table"], src, dst, moved)
            _move_rows(s["v_pool"], c["dim"], "v", s["table"], src, dst, moved)
            new = s["seq_lens"] + s["accepted"]
        return {"k": s["k_pool"].view(F8["e4m3"]), "v": s["v_pool"].view(F8["e4m3"]), "lens": new}
    if own:
        from quantized_kv_cache_quant_gb300 import spec
        k, v, ws = _handles(s)
        out = torch.empty(s["q"].shape, dtype=torch.float16, device="cuda")
        spec.fp8_tree_attention(s["q"], k, v, s["table"], s["seq_lens"], s["offsets"], s["mask"], s["max_tree"],
                                s["max_seq"], out, 0.0, ws)
        return out
    return _attention(s)


# ---------------------------------------------------------------- floors

def work(case):
    c = case
    if c["op"] == "plan":
        new = c["batch"] * (c["new_lo"] + c["new_hi"]) / 2
        # each new token's slot, request and position once; each block taken and given back: table and stack entries
        return {"bytes": 16.0 * new + 16.0 * new / BT + 40.0 * c["batch"], "flops": 0}
    if c["op"] == "append":
        return {"bytes": c["tokens"] * (c["heads"] * c["dim"] * 6.0 + 8.0), "flops": 0}
    if c["op"] == "accept":
        return {"bytes": c["batch"] * ((c["path"] / 2 if c["batch"] > 1 else c["path"]) * c["heads"] * c["dim"] * 4.0 + 16.0), "flops": 0}
    tree, ctx = (c["tree_lo"] + c["tree_hi"]) / 2, (c["ctx_lo"] + c["ctx_hi"]) / 2
    b, d = c["batch"], c["dim"]
    return {"bytes": b * (2.0 * c["heads"] * (ctx + tree) * d + 4.0 * tree * c["q_heads"] * d),
            "flops": 4.0 * b * c["q_heads"] * tree * (ctx + tree) * d}


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


def _nearest(y, fmt):
    """The format's value nearest to y (64 bits), ties to the even code, beyond the largest: the largest."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    y = y.clamp(-FMAX[fmt], FMAX[fmt])
    e = (torch.frexp(y).exponent - 1).clamp(min=low)
    step = torch.ldexp(torch.ones_like(y), e - bits)
    return (y / step).round() * step


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "plan":
        return None                                   # whole numbers: they are compared with the plain form's
    if c["op"] == "append":
        out = {}
        for name, role in (("k", "k"), ("v", "v")):
            pool, x, scale = s[name + "_pool"], s[name + "_new"], s[name + "_scale"]
            n, h, d = x.shape
            if pool.numel() > 1 << 30:
                return None
            val = _code_values(c["fmt"])[pool.view(-1).long()].view(pool.shape)
            y = _nearest(x.double() / scale.double().view(1, -1, 1), c["fmt"])
            block, row = s["slots"] // BT, s["slots"] % BT
            where = _offsets(d, role)
            for r in range(BT):                       # the tokens of row r of their blocks
                mine = row == r
                part = val[block[mine]]
                part[:, :, where[r]] = y[mine]
                val[block[mine]] = part
            out[name] = val
        return out
    if c["op"] == "accept":
        out = {"lens": None}
        paths, lens, counts, table = s["path"].tolist(), s["seq_lens"].tolist(), s["accepted"].tolist(), s["table"].tolist()
        for name in ("k", "v"):
            val = _code_values("e4m3")[s[name + "_pool"].view(-1).long()].view(s[name + "_pool"].shape)
            was, where = val.clone(), _offsets(c["dim"], name)
            for b, n in enumerate(counts):
                for i in range(n):
                    p, q = lens[b] + paths[b][i], lens[b] + i
                    val[table[b][q // BT]][:, where[q % BT]] = was[table[b][p // BT]][:, where[p % BT]]
            out[name] = val
        return out
    d, gq = c["dim"], c["q_heads"] // c["heads"]
    flops = work(case)["flops"]
    if flops > 4e12:
        return None
    val = _code_values(c["fmt"])
    offs = {"k": _offsets(d, "k"), "v": _offsets(d, "v")}
    first, lens = s["offsets"].tolist(), s["seq_lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(c["batch"]):
        n0, n1 = first[b], first[b + 1]
        t, total = n1 - n0, lens[b] + n1 - n0
        if t == 0 or total == 0:
            continue
        blocks = s["table"][b, : -(-total // BT)].long()
        bits = torch.arange(t, device="cuda")
        seen = (s["mask"][n0:n1][:, bits // 64] >> (bits % 64) & 1) == 1            # [t, t]
        for h in range(c["heads"]):
            kv = {}
            for name in ("k", "v"):
                raw = s[name + "_pool"][blocks, h][:, offs[name].reshape(-1)].reshape(-1, d)[:total]
                scale = s[name + "_scale"]
                kv[name] = val[raw.long()] * scale.double()[h if scale.numel() > 1 else 0]
            q = s["q"][n0:n1, h * gq:(h + 1) * gq].double().reshape(t * gq, d)
            x = q @ kv["k"].T / math.sqrt(d)
            x[:, lens[b]:] = torch.where(seen.repeat_interleave(gq, 0), x[:, lens[b]:], -math.inf)
            p = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
            o = p @ kv["v"] / p.sum(1, keepdim=True).clamp(min=1e-300)
            out[n0:n1, h * gq:(h + 1) * gq] = o.view(t, gq, d)
    return out
