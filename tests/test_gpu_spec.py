"""Speculative decoding over the paged FP8 cache on the GPU: tables, slots,
bytes and moved rows equal the oracle's; tree attention stays within a bound
derived from the arithmetic; the calls together follow a plain decode."""
import numpy as np
import pytest

from oracle import fp8, layout
from oracle import spec as ospec
from kvq_helpers import dev, host

pytestmark = pytest.mark.gpu

KEY, VALUE = 2, 1          # the oracle's in-block orders of the two roles


def _mods():
    from quantized_kv_cache_quant_gb300 import kvq, spec
    return kvq, spec


def i32(x):
    return dev(np.asarray(x, np.int32))


# ---------------------------------------------------------------- block tables

def _held_state(rng, batch, width, num_blocks, most):
    held = rng.integers(0, most + 1, batch)
    while held.sum() > num_blocks:
        held[rng.integers(batch)] = 0
    perm = rng.permutation(num_blocks)
    table, at = np.full((batch, width), -1, np.int32), 0
    for b, n in enumerate(held):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, held.astype(np.int32), perm[at:].tolist()


@pytest.mark.parametrize("batch,width,num_blocks,bt,most", [
    (1, 1, 1, 16, 1), (1, 7, 5, 16, 3), (3, 8, 11, 1, 4), (8, 512, 1500, 16, 250), (33, 40, 900, 32, 30),
    (256, 100, 20000, 16, 90), (1025, 17, 9000, 16, 8), (4096, 5, 12000, 16, 5), (2, 9000, 17000, 16, 8000)])
def test_resize_matches_oracle(batch, width, num_blocks, bt, most):
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(batch * 31 + width)
    table, held, free = _held_state(rng, batch, width, num_blocks, most)
    d_table, d_held, d_count = dev(table), dev(held), i32([len(free)])
    stack = np.full(num_blocks, -7, np.int32)
    stack[: len(free)] = free
    d_free, granted = dev(stack), torch.full((batch,), -1, dtype=torch.int32, device="cuda")
    for step in range(4):      # grow, shrink and mix from the state the call before left
        target = rng.integers(0, min(width, most + 3) * bt + 1, batch)
        if step == 1:
            target[rng.integers(batch)] = -1
            target[rng.integers(batch)] = width * bt + 1
            target[rng.integers(batch)] = 2**31 - 1
        if step == 2:
            target[:] = rng.integers(0, bt + 1, batch)      # mostly releases
        spec.kv_blocks_resize(d_table, d_held, i32(target), bt, d_free, d_count, granted if step != 3 else None)
        table, held, free, ok = ospec.resize(table, held, target, bt, free)
        assert np.array_equal(host(d_table), table)
        assert np.array_equal(host(d_held), held)
        assert host(d_count)[0] == len(free)
        assert np.array_equal(host(d_free)[: len(free)], free)
        if step != 3:
            assert np.array_equal(host(granted), ok)


def test_grow_and_shrink_restore_the_stack():
    kvq, spec = _mods()
    t = spec.BlockTables(5, 20, 60)
    first = host(t.free_blocks).copy()
    t.resize(i32([17, 0, 300, 1, 33]))
    assert host(t.n_held).tolist() == [2, 0, 19, 1, 3] and host(t.granted).tolist() == [1] * 5
    assert sorted(host(t.table)[host(t.table) >= 0].tolist()) == list(range(25))
    t.resize(i32([0] * 5))
    assert np.array_equal(host(t.free_blocks), first) and host(t.free_count)[0] == 60
    assert (host(t.table) == -1).all()


def test_resize_of_the_largest_table():
    """2^31 - 1 entries: all released, then granted again."""
    import torch
    _, spec = _mods()
    n = 2 ** 31 - 1
    table = torch.arange(n, dtype=torch.int32, device="cuda").view(1, n)
    free = torch.zeros(n, dtype=torch.int32, device="cuda")
    held, count = i32([n]), i32([0])
    spec.kv_blocks_resize(table, held, i32([0]), 1, free, count)
    assert (int(held), int(count)) == (0, n)
    assert int(table.max()) == -1 and int(table.min()) == -1
    for at in (0, 1, 65535, n // 2, n - 65536, n - 1):
        assert int(free[at]) == n - 1 - at             # the first one released is on top
    spec.kv_blocks_resize(table, held, i32([n]), 1, free, count)
    assert (int(held), int(count)) == (n, 0)
    want = torch.arange(n, dtype=torch.int32, device="cuda")
    assert torch.equal(table[0], want)


def test_resize_with_a_state_that_does_not_add_up_stays_inside():
    """More blocks held and free than the pool has: the stack never runs past its end."""
    kvq, spec = _mods()
    table = dev(np.zeros((4, 8), np.int32))
    held, count = i32([8, 99, 8, -3]), i32([50])
    free = dev(np.arange(20, dtype=np.int32))
    spec.kv_blocks_resize(table, held, i32([0, 0, 0, 16]), 16, free, count)
    assert host(count)[0] <= 20 and host(held).tolist()[:3] == [0, 0, 0]


# ---------------------------------------------------------------- slot map

@pytest.mark.parametrize("batch,width,num_blocks,bt,top,spare", [
    (1, 4, 9, 16, 5, 0), (1, 4, 9, 16, 1, 3), (8, 30, 100, 16, 8, 5), (300, 12, 700, 16, 40, 1), (5, 900, 5000, 16, 6000, 2),
    (4096, 3, 9000, 1, 3, 0), (7, 6, 50, 32, 100, 9)])
def test_slot_map_matches_oracle(batch, width, num_blocks, bt, top, spare):
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(batch + width)
    table = rng.integers(-2, num_blocks + 2, (batch, width)).astype(np.int32)     # some entries outside the pool
    seq = rng.integers(0, width * bt, batch)
    new = rng.integers(-1, top + 1, batch)                                        # negative: none; some past the table
    total = int(np.maximum(new, 0).sum())
    for rows in (max(1, total + spare), max(1, total // 2 + 1)):
        off = torch.empty(batch + 1, dtype=torch.int32, device="cuda")
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        ids, pos = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(2))
        spec.kv_slot_map(dev(table), i32(seq), i32(new), bt, num_blocks, off, slots, ids, pos)
        want = ospec.slot_map(table, seq, new, bt, num_blocks, rows)
        for got, w in zip((off, slots, ids, pos), want):
            assert np.array_equal(host(got), w)
        only = torch.empty_like(slots)
        spec.kv_slot_map(dev(table), i32(seq), i32(new), bt, num_blocks, off, only)
        assert torch.equal(only, slots)


# ---------------------------------------------------------------- pools

class Pools:
    """A key and a value pool on the device with their natural bytes on the host."""

    def __init__(self, rng, blocks, heads, dim, fmt, per_head, fill=None):
        import torch
        kvq, _ = _mods()
        self.fmt, self.nat, self.pool, self.scale = fmt, [], [], []
        for role, order in ((kvq.ROLE_KEY, KEY), (kvq.ROLE_VALUE, VALUE)):
            sc = rng.uniform(0.005, 0.02, heads if per_head else 1).astype(np.float32)
            x = rng.standard_normal((blocks, heads, 16, dim)).astype(np.float16)
            nat = fp8.quantize(x.transpose(1, 0, 2, 3).reshape(1, heads, -1, dim), sc if per_head else sc[0], fmt)
            nat = np.ascontiguousarray(nat.reshape(heads, blocks, 16, dim).transpose(1, 0, 2, 3))
            if fill is not None:
                nat[:] = fill
            p = kvq.Fp8Pool(role, blocks, heads, dim, kvq.FP8_FORMATS[fmt], per_head)
            p.scale.copy_(torch.from_numpy(sc))
            self.nat.append(nat)
            self.pool.append(p)
            self.scale.append(sc)
        self.upload()

    def upload(self):
        import torch
        for nat, p, order in zip(self.nat, self.pool, (KEY, VALUE)):
            p.view().copy_(torch.from_numpy(layout.fp8_pack_pool(nat, order)))

    def check(self):
        for nat, p, order, name in zip(self.nat, self.pool, (KEY, VALUE), "kv"):
            got = host(p.view())
            want = layout.fp8_pack_pool(nat, order)
            assert np.array_equal(got, want), f"{name}: {np.sum(got != want)} bytes differ"

    @property
    def descs(self):
        return self.pool[0].desc, self.pool[1].desc


@pytest.mark.parametrize("fmt,per_head", [("e4m3", False), ("e5m2", True)])
@pytest.mark.parametrize("heads,dim,n,kind", [
    (1, 64, 1, "random"), (2, 128, 7, "random"), (3, 64, 40, "runs"), (8, 128, 33, "runs"), (8, 64, 2000, "runs"),
    (8, 128, 3000, "random"), (5, 128, 2500, "long"), (2, 64, 19, "long")])
def test_append_bytes(fmt, per_head, heads, dim, n, kind):
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(n * heads + dim)
    blocks = n // 4 + 12
    if kind == "random":
        slots = rng.permutation(blocks * 16)[:n]
    else:
        perm, slots = rng.permutation(blocks), []
        at = 0
        while len(slots) < n:        # runs that start and end inside blocks
            run, r0 = (int(rng.integers(1, 20)), int(rng.integers(0, 16))) if kind == "runs" else (n, 5)
            need = -(-(r0 + run) // 16)
            if at + need > blocks:
                break
            p = np.arange(r0, r0 + run)
            slots += (perm[at + p // 16] * 16 + p % 16).tolist()
            at += need
        slots = np.array(slots[:n])
        n = len(slots)
    slots = slots.astype(np.int64)
    skip = rng.random(n) < 0.1
    slots[skip] = rng.choice([-1, -5, blocks * 16, blocks * 16 + 3, 2**40], skip.sum())
    p = Pools(rng, blocks, heads, dim, fmt, per_head)
    x = rng.standard_normal((2, n, heads, dim)).astype(np.float16) * np.float16(2.0)
    x[0, 0, 0, :6] = [np.nan, np.inf, -np.inf, -0.0, 65504.0, 1e-7]
    x[1, n // 2, -1, -6:] = [np.nan, np.inf, -np.inf, -0.0, -65504.0, 6e-8]
    # rows of a wider buffer, as a fused projection gives them
    wide = torch.zeros((n, (2 * heads + 3) * dim), dtype=torch.float16, device="cuda")
    kn = wide[:, dim: (heads + 1) * dim].unflatten(1, (heads, dim))
    vn = wide[:, (heads + 2) * dim: (2 * heads + 2) * dim].unflatten(1, (heads, dim))
    kn.copy_(dev(x[0]))
    vn.copy_(dev(x[1]))
    spec.fp8_kv_append(*p.descs, kn, vn, dev(slots))
    for r in range(2):
        p.nat[r] = ospec.append(p.nat[r], x[r], slots, p.scale[r] if per_head else p.scale[r][0], fmt)
    p.check()


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -120, 2.0 ** 100, 0.0])
def test_append_extreme_scales(scale):
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(3)
    p = Pools(rng, 4, 2, 64, "e4m3", False)
    x = rng.standard_normal((20, 2, 64)).astype(np.float16)
    x[3, 1, 5] = 0
    for r in range(2):
        p.scale[r][:] = scale
        p.pool[r].scale.fill_(scale)
        with np.errstate(all="ignore"):
            p.nat[r] = ospec.append(p.nat[r], x, np.arange(9, 29), p.scale[r][0], "e4m3")
    spec.fp8_kv_append(*p.descs, dev(x), dev(x), dev(np.arange(9, 29)))
    p.check()


@pytest.mark.parametrize("heads,dim,batch,tree,plen", [(1, 64, 1, 1, 1), (2, 128, 3, 20, 7), (8, 128, 40, 64, 12),
                                                       (3, 64, 5, 256, 256), (16, 128, 2, 33, 9)])
def test_accept_moves_rows(heads, dim, batch, tree, plen):
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(tree + heads)
    seq = rng.integers(0, 50, batch)
    width = -(-(50 + tree) // 16)
    table = rng.permutation(batch * width + 3)[: batch * width].reshape(batch, width).astype(np.int32)
    p = Pools(rng, batch * width + 3, heads, dim, "e4m3", False)
    path = np.sort(np.argsort(rng.random((batch, tree)), 1)[:, :plen], 1).astype(np.int32)
    acc = rng.integers(0, plen + 1, batch)
    acc[0] = plen
    new = torch.empty(batch, dtype=torch.int32, device="cuda")
    spec.fp8_kv_accept(*p.descs, dev(table), i32(seq), dev(path), i32(acc), new)
    for r in range(2):
        p.nat[r] = ospec.accept(p.nat[r], table, seq, path, acc)
    p.check()
    assert np.array_equal(host(new), seq + acc)
    # lengths advanced in place; rows already in place are left alone
    lens = i32(seq)
    spec.fp8_kv_accept(*p.descs, dev(table), lens, i32(np.tile(np.arange(plen), (batch, 1))), i32(acc), lens)
    p.check()
    assert np.array_equal(host(lens), seq + acc)


def test_accept_of_lengths_beyond_every_table():
    """Lengths up to 2^31 - 1 behind the table: nothing moves, and the call's work does not follow them."""
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(7)
    p = Pools(rng, 4, 2, 64, "e4m3", False)
    p.upload()
    path = np.tile(np.arange(1, 201, dtype=np.int32), (3, 1))
    lens = np.array([2 ** 31 - 1, 2 ** 31 - 150, 65], np.int32)
    new = torch.zeros(3, dtype=torch.int32, device="cuda")
    spec.fp8_kv_accept(*p.descs, i32([[0, 1, 2, 3]] * 3), dev(lens), dev(path), i32([200] * 3), new)
    assert host(new).tolist() == [int(np.int32((int(n) + 200 + 2 ** 31) % 2 ** 32 - 2 ** 31)) for n in lens]
    p.check()


def test_accept_skips_what_is_outside():
    kvq, spec = _mods()
    rng = np.random.default_rng(5)
    p = Pools(rng, 3, 1, 64, "e4m3", False)
    table = i32([[0, 7], [2, -1]])                     # entries outside the pool
    lens = i32([14, 3])
    spec.fp8_kv_accept(*p.descs, table, lens, i32([[1, 4], [-1, 300]]), i32([2, 9]), lens)
    want = [n.copy() for n in p.nat]
    for n, w in zip(p.nat, want):
        w[0, :, 14] = n[0, :, 15]
    p.nat = want
    p.check()
    assert host(lens).tolist() == [16, 5]


# ---------------------------------------------------------------- tree attention

def random_sees(rng, trees, full=False):
    n = int(sum(trees))
    sees = np.zeros((n, max(trees) if len(trees) else 1), bool)
    at = 0
    for t in trees:
        for i in range(t):
            if full:
                sees[at + i, :i + 1] = True
            else:
                par = i - int(rng.integers(1, 5))
                if par >= 0:
                    sees[at + i] = sees[at + par]
                sees[at + i, i] = True
        at += t
    return sees


def tree_bound(mag, spread, dots, ref, wide, dim):
    """|error| of the kernel's output. Scores are fp32 sums of dim products
    (error at most dim * 2^-24 * sum |q k| * scale, and as much again for the
    scale, the subtraction of the maximum and ex2), which moves a weight by that
    relative amount; sums over tokens and the division add a few 2^-24 more.
    Weights rounded to fp16 add 2^-11 relative (2^-22 when kept in two parts)
    and at most 2^-25 of the largest weight where they are subnormal; an fp16
    output adds half a step."""
    rel = 4 * dim * 2.0 ** -24 * dots[..., None] + 2.0 ** -16 + (2.0 ** -21 if wide else 2.0 ** -11)
    out = rel * mag + 2.0 ** -24 * spread
    if not wide:
        out = out + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25
    return out


# max_seq_len of every call, where it is more than the lengths need: calls with short tables and few rows take one kernel,
# the same ones with long tables another
LONGEST = [0]


@pytest.fixture
def long_tables():
    LONGEST[0] = 4096
    yield
    LONGEST[0] = 0


def run_tree(spec, p, table, seq, trees, sees, q, wide, max_tree=None, extra_rows=0, strided=False, ws=None, scale=0.0):
    import torch
    n, hq, d = q.shape
    off = np.concatenate([[0], np.cumsum(trees)]).astype(np.int32)
    max_tree = max_tree or max(1, max(trees))
    words = -(-max_tree // 64)
    padded = np.zeros((n + extra_rows, words * 64), bool)
    padded[:n, : sees.shape[1]] = sees
    mask = spec.pack_tree_mask(dev(padded)).contiguous()
    qq = np.concatenate([q, np.full((extra_rows, hq, d), np.nan, np.float16)])
    if strided:
        buf = torch.full((n + extra_rows, (hq + 2) * d), float("nan"), dtype=torch.float16, device="cuda")
        dq = buf[:, d:(hq + 1) * d].unflatten(1, (hq, d))
        dq.copy_(dev(qq))
    else:
        dq = dev(qq)
    out = torch.full((n + extra_rows, hq, d), -77.0, dtype=torch.float32 if wide else torch.float16, device="cuda")
    if ws is None:
        ws = spec.tree_workspace(len(seq), p.descs[0].kv_heads, hq, d, max_tree)
    if table.shape[1] * 16 < LONGEST[0]:
        table = np.pad(table, ((0, 0), (0, LONGEST[0] // 16 - table.shape[1])), constant_values=-1)
    width = table.shape[1]
    most = max(int(max(s + t for s, t in zip(seq, trees))), LONGEST[0])
    spec.fp8_tree_attention(dq, *p.descs, dev(table), i32(seq), dev(off), mask, max_tree, max(1, min(most, width * 16)), out,
                            scale, ws)
    got = host(out).astype(np.float64)
    assert (got[n:] == -77.0).all()                    # rows behind the last node are left as they were
    assert int(ws[:4].view(torch.int32).item()) == 0   # no wait ran out
    return got[:n], off


def check_tree(rng, heads, gq, dim, seq, trees, fmt="e4m3", per_head=False, wide=False, sees=None, **kw):
    kvq, spec = _mods()
    width = max(1, -(-max(s + t for s, t in zip(seq, trees)) // 16))
    blocks = sum(-(-(s + t) // 16) for s, t in zip(seq, trees)) + 2
    perm = rng.permutation(blocks)
    table, at = np.full((len(seq), width), -1, np.int32), 0
    for b, (s, t) in enumerate(zip(seq, trees)):
        m = -(-(s + t) // 16)
        table[b, :m] = perm[at:at + m]
        at += m
    p = Pools(rng, blocks, heads, dim, fmt, per_head)
    for b, (s, t) in enumerate(zip(seq, trees)):       # stale NaN rows behind the last node
        if (s + t) % 16:
            for nat in p.nat:
                nat[table[b, (s + t) // 16], :, (s + t) % 16:] = 0x7F
    # blocks of nobody hold NaN too
    for nat in p.nat:
        nat[perm[at:]] = 0x7F
    p.upload()
    sees = random_sees(rng, trees) if sees is None else sees
    q = rng.standard_normal((int(sum(trees)), heads * gq, dim)).astype(np.float16)
    got, off = run_tree(spec, p, table, seq, trees, sees, q, wide, **kw)
    scale = np.float32(kw.get("scale") or np.float32(1.0) / np.sqrt(np.float32(dim)))
    ref, mag, spread, dots = ospec.tree_attention(q, p.nat[0], p.nat[1], p.scale[0], p.scale[1], fmt, table, seq, off, sees,
                                                  scale)
    err, tol = np.abs(got - ref), tree_bound(mag, spread, dots, ref, wide, dim)
    assert np.all(err <= tol), f"worst {np.max(err / np.maximum(tol, 1e-30)):.3g} of the bound, abs {err.max():.3g}"


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dim,fmt,per_head", [(128, "e4m3", False), (64, "e4m3", True), (128, "e5m2", True), (64, "e5m2", False)])
@pytest.mark.parametrize("heads,gq,seq,trees", [
    (1, 1, [0], [1]),                                  # one node, nothing before it
    (2, 4, [17], [5]),
    (2, 8, [100, 3, 0, 250], [1, 4, 7, 2]),            # few rows a kv head
    (1, 4, [129, 64, 15], [9, 8, 16]),                 # 32 to 64 rows
    (2, 2, [300, 0, 1, 16, 31], [33, 20, 0, 1, 40]),   # a request without nodes among others
    (1, 8, [511, 40], [63, 17]),                       # several row tiles
    (1, 1, [70], [130]),                               # three mask words
])
def test_tree_matches_oracle(heads, gq, seq, trees, dim, fmt, per_head, wide):
    check_tree(np.random.default_rng(dim + gq + len(seq)), heads, gq, dim, seq, trees, fmt, per_head, wide)


@pytest.mark.parametrize("gq", [3, 5, 7, 16, 64])
def test_tree_odd_head_groups(gq):
    check_tree(np.random.default_rng(gq), 2 if gq < 16 else 1, gq, 128, [37, 90], [5, 11])


@pytest.mark.parametrize("seq", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 1023])
def test_tree_context_lengths(seq):
    check_tree(np.random.default_rng(seq), 1, 4, 128, [seq], [6], wide=True)
    check_tree(np.random.default_rng(seq), 1, 4, 64, [seq, max(0, seq - 1)], [17, 31])


def test_tree_long_context_is_split():
    check_tree(np.random.default_rng(9), 2, 4, 128, [6000, 100], [3, 5], wide=True)
    check_tree(np.random.default_rng(10), 1, 8, 64, [5001], [20])


def test_tree_many_requests():
    rng = np.random.default_rng(11)
    check_tree(rng, 2, 2, 64, rng.integers(0, 60, 300).tolist(), rng.integers(0, 6, 300).tolist())


def test_tree_of_256_nodes():
    check_tree(np.random.default_rng(12), 1, 2, 64, [40], [256])


def test_tree_rows_that_see_nothing_are_zero():
    rng = np.random.default_rng(13)
    sees = random_sees(rng, [20, 20])
    sees[3] = False
    sees[21] = False
    sees[25, :] = True
    check_tree(rng, 2, 4, 128, [0, 0], [20, 20], sees=sees)
    check_tree(rng, 1, 1, 64, [0, 0], [20, 20], sees=sees, wide=True)
    check_tree(rng, 2, 4, 64, [0, 0], [20, 20], sees=np.zeros((40, 20), bool))


@pytest.mark.parametrize("gq", [1, 8])
@pytest.mark.parametrize("dim", [64, 128])
def test_tree_nan_in_masked_nodes_stays_there(dim, gq):
    """Node 2's keys and node 4's values are NaN: rows that do not see them are finite and right, rows that do are NaN."""
    kvq, spec = _mods()
    rng = np.random.default_rng(14)
    seq, trees = [30, 5], [9, 9]
    table = np.array([[3, 1, 0], [2, 4, -1]], np.int32)
    p = Pools(rng, 5, 1, dim, "e4m3", False)
    sees = random_sees(rng, trees)
    sees[:, 2] = sees[:, 4] = False
    sees[2, 2] = sees[4, 4] = sees[11, 2] = sees[13, 4] = True
    for b in range(2):
        for node, nat in ((2, p.nat[0]), (4, p.nat[1])):
            pos = seq[b] + node
            nat[table[b, pos // 16], :, pos % 16, :] = 0xFF
    p.upload()
    q = rng.standard_normal((18, gq, dim)).astype(np.float16)
    for wide in (False, True):
        got, off = run_tree(spec, p, table, seq, trees, sees, q, wide)
        ref, mag, spread, dots = ospec.tree_attention(q, p.nat[0], p.nat[1], p.scale[0], p.scale[1], "e4m3", table, seq, off,
                                                      sees, np.float32(1.0) / np.sqrt(np.float32(dim)))
        clean = [i for i in range(18) if i not in (2, 4, 11, 13)]
        assert np.isnan(got[[2, 4, 11, 13]]).all() and np.isnan(ref[[2, 4, 11, 13]]).all()
        assert np.all(np.abs(got - ref)[clean] <= tree_bound(mag, spread, dots, ref, wide, dim)[clean])


def test_tree_nan_channel_of_a_seen_node_reaches_its_channel_only():
    kvq, spec = _mods()
    rng = np.random.default_rng(15)
    p = Pools(rng, 2, 1, 64, "e5m2", False)
    p.nat[1][1, 0, 3, 17] = 0x7F                       # node 3 of a tree without context, channel 17
    p.upload()
    sees = np.tril(np.ones((6, 6), bool))
    sees[5, 3] = False
    q = rng.standard_normal((6, 2, 64)).astype(np.float16)
    got, _ = run_tree(spec, p, np.array([[1]], np.int32), [0], [6], sees, q, True)
    bad = np.isnan(got)
    assert bad[3:5, :, 17].all() and bad.sum() == 4


def test_tree_query_nan_stays_in_its_row():
    kvq, spec = _mods()
    rng = np.random.default_rng(16)
    p = Pools(rng, 4, 1, 128, "e4m3", False)
    sees = random_sees(rng, [8])
    q = rng.standard_normal((8, 8, 128)).astype(np.float16)
    clean, _ = run_tree(spec, p, np.array([[0, 1, 2]], np.int32), [25], [8], sees, q, False)
    q[3, 5, 7] = np.nan
    got, _ = run_tree(spec, p, np.array([[0, 1, 2]], np.int32), [25], [8], sees, q, False)
    assert np.isnan(got[3, 5]).all()
    got[3, 5] = clean[3, 5]
    assert np.array_equal(got, clean)


def test_tree_strided_queries_and_padded_rows():
    check_tree(np.random.default_rng(17), 2, 4, 128, [200, 31], [7, 12], extra_rows=9, strided=True)
    check_tree(np.random.default_rng(18), 2, 1, 64, [200, 31], [7, 2], extra_rows=1, strided=True, wide=True, max_tree=70)


def test_tree_softmax_scale_and_large_scores():
    check_tree(np.random.default_rng(19), 1, 8, 128, [400], [9], scale=0.7)
    check_tree(np.random.default_rng(20), 1, 2, 64, [300], [40], scale=2.0, wide=True)


def test_tree_rising_scores():
    """Each later token scores higher than the ones before: the running maximum moves in every tile."""
    kvq, spec = _mods()
    rng = np.random.default_rng(21)
    for dim, gq in ((128, 1), (64, 16)):
        p = Pools(rng, 70, 1, dim, "e4m3", False)
        ramp = np.linspace(-4, 4, 70 * 16, dtype=np.float32)[:, None] * np.ones(dim, np.float32)
        p.nat[0] = fp8.quantize(ramp.astype(np.float16).reshape(70, 1, 16, dim), p.scale[0][0], "e4m3")
        p.upload()
        table, seq, trees = np.arange(70, dtype=np.int32)[None], [70 * 16 - 12], [12]
        sees = random_sees(rng, trees)
        q = (0.3 + 0.01 * rng.standard_normal((12, gq, dim))).astype(np.float16)
        for wide in (False, True):
            got, off = run_tree(spec, p, table, seq, trees, sees, q, wide)
            ref, mag, spread, dots = ospec.tree_attention(q, *p.nat, *p.scale, "e4m3", table, seq, off, sees,
                                                          np.float32(1.0) / np.sqrt(np.float32(dim)))
            assert np.all(np.abs(got - ref) <= tree_bound(mag, spread, dots, ref, wide, dim))


def test_tree_bad_tables_and_lengths_stay_inside():
    """Entries outside the pool, lengths past the table and offsets out of order give some numbers, no fault."""
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(22)
    p = Pools(rng, 3, 2, 128, "e4m3", False)
    q = dev(rng.standard_normal((6, 8, 128)).astype(np.float16))
    mask = torch.full((6, 1), -1, dtype=torch.int64, device="cuda")
    ws = spec.tree_workspace(3, 2, 8, 128, 4)
    out = torch.zeros((6, 8, 128), dtype=torch.float16, device="cuda")
    for off in ([0, 3, 2, 50], [-4, 2, 9, 9], [0, 2, 4, 6]):
        spec.fp8_tree_attention(q, *p.descs, i32([[5, -1], [0, 99], [1, 2]]), i32([1000, -5, 31]), i32(off), mask, 4, 32, out,
                                0.0, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0


def test_tree_one_node_matches_decode():
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(23)
    b, h, hq, d = 3, 2, 16, 128
    p = Pools(rng, 40, h, d, "e4m3", False)
    table = rng.permutation(36).reshape(3, 12).astype(np.int32)
    lens = [150, 1, 77]
    q = rng.standard_normal((b, hq, d)).astype(np.float16)
    got, _ = run_tree(spec, p, table, [n - 1 for n in lens], [1, 1, 1], np.ones((3, 1), bool), q, True)
    out = torch.empty((b, hq, d), dtype=torch.float32, device="cuda")
    n = kvq.fp8_decode_workspace_bytes(b, hq, d)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    kvq.fp8_decode_attention(dev(q), *p.descs, dev(table), i32(lens), b, hq, 12, 192, out, True, 0.0, ws, n)
    assert np.abs(got - host(out)).max() <= 2e-5       # both a few 1e-6 from the 64-bit result on unit-size values


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dim", [64, 128])
def test_decode_after_append_does_not_read_stale_rows(dim, fmt):
    """A cache filled by appends alone, in blocks that held NaN before: the rows behind each sequence stay as they were,
    and the single-token decode does not see them either."""
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(33)
    b, h, hq, lens = 3, 2, 8, [1, 19, 45]
    p = Pools(rng, 12, h, dim, fmt, False, fill=0x7F)
    table = rng.permutation(12)[:9].reshape(3, 3).astype(np.int32)
    new = torch.empty(sum(lens), dtype=torch.int64, device="cuda")
    off = torch.empty(b + 1, dtype=torch.int32, device="cuda")
    spec.kv_slot_map(dev(table), i32([0] * b), i32(lens), 16, 12, off, new)
    x = rng.standard_normal((2, sum(lens), h, dim)).astype(np.float16)
    spec.fp8_kv_append(*p.descs, dev(x[0]), dev(x[1]), new)
    q = rng.standard_normal((b, hq, dim)).astype(np.float16)
    out = torch.empty((b, hq, dim), dtype=torch.float32, device="cuda")
    n = kvq.fp8_decode_workspace_bytes(b, hq, dim)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for q_fp8 in (False, True):
        kvq.fp8_decode_attention(dev(q), *p.descs, dev(table), i32(lens), b, hq, 3, 48, out, True, 0.0, ws, n, q_fp8=q_fp8)
        got = host(out)
        qq = fp8.query_hat(*fp8.quantize_query(q)) if q_fp8 else q.astype(np.float64)
        at = 0
        for bi, m in enumerate(lens):
            kk, vv = (fp8.decode(fp8.quantize(x[r, at:at + m].transpose(1, 0, 2)[None], p.scale[r][0], fmt)[0], fmt) *
                      np.float64(p.scale[r][0]) for r in range(2))
            at += m
            for g in range(hq):
                s = kk[g // 4] @ qq[bi, g] / np.sqrt(dim)
                w = np.exp(s - s.max())
                assert np.abs(got[bi, g] - w @ vv[g // 4] / w.sum()).max() <= 2e-3


def test_tree_same_call_twice_gives_the_same_bits():
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(24)
    p = Pools(rng, 300, 2, 128, "e4m3", False)
    table = rng.permutation(300)[:280].reshape(1, 280).astype(np.int32)
    sees, q = random_sees(rng, [16]), rng.standard_normal((16, 8, 128)).astype(np.float16)
    ws = spec.tree_workspace(1, 2, 8, 128, 16)
    a, _ = run_tree(spec, p, table, [4400], [16], sees, q, True, ws=ws)
    for _ in range(3):
        b, _ = run_tree(spec, p, table, [4400], [16], sees, q, True, ws=ws)
        assert np.array_equal(a, b)


TREE_SHAPES = [(2, 4, [17], [5]), (2, 8, [100, 3, 0, 250], [1, 4, 7, 2]), (1, 4, [129, 64, 15], [9, 8, 16]),
               (2, 2, [300, 0, 1, 16, 31], [33, 20, 0, 1, 40]), (1, 8, [511, 40], [63, 17]), (1, 1, [70], [130])]


@pytest.mark.parametrize("test,args", [(test_tree_matches_oracle, s + f + (w,)) for s in TREE_SHAPES for w in (False, True)
                                       for f in ((128, "e4m3", False), (64, "e5m2", True))]
                         + [(test_tree_odd_head_groups, (g,)) for g in (3, 7, 64)]
                         + [(test_tree_context_lengths, (n,)) for n in (1, 15, 16, 63, 64, 65, 129, 1023)]
                         + [(test_tree_nan_in_masked_nodes_stays_there, (d, 8)) for d in (64, 128)]
                         + [(t, ()) for t in (test_tree_rows_that_see_nothing_are_zero, test_tree_query_nan_stays_in_its_row,
                                              test_tree_strided_queries_and_padded_rows, test_tree_many_requests,
                                              test_tree_softmax_scale_and_large_scores, test_tree_rising_scores,
                                              test_tree_of_256_nodes, test_tree_same_call_twice_gives_the_same_bits)])
def test_tree_with_long_tables(long_tables, test, args):
    test(*args)


def test_tree_more_requests_than_threads_of_a_block(long_tables):
    rng = np.random.default_rng(29)
    check_tree(rng, 1, 4, 64, rng.integers(0, 40, 700).tolist(), rng.integers(0, 7, 700).tolist())


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dim,fmt", [(128, "e4m3"), (64, "e5m2")])
@pytest.mark.parametrize("seq,trees", [
    ([700, 0, 65, 130, 1], [90, 80, 64, 70, 100]),     # the longest passes every ring of tiles more than twice
    ([40] * 12, [20, 33, 40, 64, 17, 31, 50, 63, 21, 40, 35, 64]),  # more pairs than blocks
])
def test_tree_of_many_rows(seq, trees, dim, fmt, wide):
    """Trees with more rows than one stream of the tensor cores' kernel, in enough requests that it takes its wide tiles."""
    check_tree(np.random.default_rng(dim + len(seq)), 8, 8, dim, seq, trees, fmt, True, wide)


@pytest.mark.parametrize("dim,wide", [(128, False), (128, True), (64, False)])
def test_tree_many_rows_see_nan_nodes_only_where_the_mask_says(dim, wide):
    kvq, spec = _mods()
    rng = np.random.default_rng(26)
    seq, trees = [30, 5, 90, 0], [80, 81, 82, 79]
    sees, at = random_sees(rng, trees), np.cumsum([0] + trees)
    table = np.full((4, 12), -1, np.int32)
    perm, used = rng.permutation(40), 0
    for b in range(4):
        m = -(-(seq[b] + trees[b]) // 16)
        table[b, :m], used = perm[used:used + m], used + m
    p = Pools(rng, 40, 8, dim, "e4m3", False)
    sees[:, 2] = sees[:, 70] = False
    for b in range(4):
        sees[at[b] + 2, 2] = sees[at[b] + 70, 70] = True
        for node, nat in ((2, p.nat[0]), (70, p.nat[1])):
            pos = seq[b] + node
            nat[table[b, pos // 16], :, pos % 16, :] = 0xFF
    p.upload()
    n = int(at[-1])
    q = rng.standard_normal((n, 64, dim)).astype(np.float16)
    got, off = run_tree(spec, p, table, seq, trees, sees, q, wide)
    ref, mag, spread, dots = ospec.tree_attention(q, p.nat[0], p.nat[1], p.scale[0], p.scale[1], "e4m3", table, seq, off, sees,
                                                  np.float32(1.0) / np.sqrt(np.float32(dim)))
    dirty = [at[b] + i for b in range(4) for i in (2, 70)]
    clean = [i for i in range(n) if i not in dirty]
    assert np.isnan(got[dirty]).all() and np.isnan(ref[dirty]).all()
    assert np.all(np.abs(got - ref)[clean] <= tree_bound(mag, spread, dots, ref, wide, dim)[clean])


@pytest.mark.parametrize("heads,gq,nodes", [(2, 8, 8), (8, 8, 200)])
def test_tree_bad_tables_and_lengths_of_wide_trees_stay_inside(heads, gq, nodes):
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(27)
    p = Pools(rng, 3, heads, 128, "e4m3", False)
    n = 3 * nodes
    q = dev(rng.standard_normal((n, heads * gq, 128)).astype(np.float16))
    mask = torch.full((n, -(-nodes // 64)), -1, dtype=torch.int64, device="cuda")
    ws = spec.tree_workspace(3, heads, heads * gq, 128, nodes)
    out = torch.zeros((n, heads * gq, 128), dtype=torch.float16, device="cuda")
    table = torch.full((3, 256), -1, dtype=torch.int32, device="cuda")
    table[1:, 1] = 99
    for off in ([0, nodes, 2, 50 * n], [-4, 2, n + 3, n + 3], [0, nodes, 2 * nodes, n]):
        for lens in ([100000, -5, 31], [0, 0, 0], [4095, 4096, 2 ** 31 - 1]):
            spec.fp8_tree_attention(q, *p.descs, table, i32(lens), i32(off), mask, nodes, 4096, out, 0.0, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) == 0


@pytest.mark.parametrize("nodes", [2, 30, 70])
def test_tree_calls_on_two_streams_and_in_two_graphs(nodes):
    """Two calls at a time with a workspace each, eager and captured, give what one call alone gives."""
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(28 + nodes)
    p = Pools(rng, 2100, 4, 128, "e4m3", False)
    table = rng.permutation(2100)[:2064].reshape(4, 516).astype(np.int32)
    sees = random_sees(rng, [nodes] * 4)
    mask = spec.pack_tree_mask(dev(np.pad(sees, ((0, 0), (0, -nodes % 64))))).contiguous()
    q = [dev(rng.standard_normal((4 * nodes, 32, 128)).astype(np.float16)) for _ in range(2)]
    lens, off, dt = i32([8000, 100, 5000, 777]), i32([0, nodes, 2 * nodes, 3 * nodes, 4 * nodes]), dev(table)
    out = [torch.zeros_like(x) for x in q]
    ws = [spec.tree_workspace(4, 4, 32, 128, nodes) for _ in range(2)]

    def call(i):
        spec.fp8_tree_attention(q[i], *p.descs, dt, lens, off, mask, nodes, 8256, out[i], 0.0, ws[i])

    want = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        want.append(out[i].clone())
        out[i].zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for i in range(2):
        streams[i].wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            call(i)
        graphs.append(g)
    for replayed in (False, True):
        for _ in range(4):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay() if replayed else call(i)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i], want[i])
            out[i].zero_()
        torch.cuda.synchronize()


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dim,nodes", [(128, 30), (128, 70), (128, 200), (64, 70)])
def test_tree_many_calls_give_the_same_bits(dim, nodes, wide):
    """A tile that is overwritten while it is read shows now and then only."""
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(30 + nodes)
    p = Pools(rng, 2100, 4, dim, "e4m3", False)
    table = dev(rng.permutation(2100)[:2064].reshape(4, 516).astype(np.int32))
    sees = random_sees(rng, [nodes] * 4)
    mask = spec.pack_tree_mask(dev(np.pad(sees, ((0, 0), (0, -nodes % 64))))).contiguous()
    q = dev(rng.standard_normal((4 * nodes, 32, dim)).astype(np.float16))
    lens, off = i32([8000, 100, 5000, 777]), i32([nodes * i for i in range(5)])
    ws = spec.tree_workspace(4, 4, 32, dim, nodes)
    out = [torch.empty(q.shape, dtype=torch.float32 if wide else torch.float16, device="cuda") for _ in range(60)]
    for o in out:
        spec.fp8_tree_attention(q, *p.descs, table, lens, off, mask, nodes, 8256, o, 0.0, ws)
    differ = sum(not torch.equal(o, out[0]) for o in out)
    assert differ == 0, f"{differ} of 60 differ"


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("fmt,dim,captured", [("e4m3", 128, False), ("e5m2", 64, False), ("e4m3", 128, True)])
def test_speculative_steps_follow_plain_decode(fmt, dim, captured):
    """Steps of draft, verify, accept over growing sequences: the cache holds what a plain decode of the accepted
    tokens would have written, the verified rows' outputs are that decode's, and rejected blocks return. Captured:
    one step as a graph, replayed with new lengths, trees and paths in the same buffers."""
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(30)
    b, h, gq, t = 3, 2, 4, 9
    hq = h * gq
    prompt = np.array([20, 1, 37])
    steps = 4
    tables = spec.BlockTables(b, 8, 40)
    p = Pools(rng, 40, h, dim, fmt, False)
    lens, off = i32(prompt), torch.zeros(b + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(b * t, dtype=torch.int64, device="cuda")

    tokens = [rng.standard_normal((2, n, h, dim)).astype(np.float16) for n in prompt]   # accepted keys, values
    first = torch.empty(int(prompt.sum()), dtype=torch.int64, device="cuda")
    tables.resize(lens)
    tables.slot_map(i32([0] * b), lens, off, first)
    flat = np.concatenate(tokens, 1)
    spec.fp8_kv_append(*p.descs, dev(flat[0]), dev(flat[1]), first)

    q = torch.zeros((b * t, hq, dim), dtype=torch.float16, device="cuda")
    kn, vn = (torch.zeros((b * t, h, dim), dtype=torch.float16, device="cuda") for _ in range(2))
    nodes, grown = torch.zeros(b, dtype=torch.int32, device="cuda"), torch.zeros(b, dtype=torch.int32, device="cuda")
    mask = torch.zeros((b * t, 1), dtype=torch.int64, device="cuda")
    path = torch.zeros((b, 4), dtype=torch.int32, device="cuda")
    acc = torch.zeros(b, dtype=torch.int32, device="cuda")
    out = torch.zeros((b * t, hq, dim), dtype=torch.float32, device="cuda")
    ws = spec.tree_workspace(b, h, hq, dim, t)

    def step():
        torch.add(lens, nodes, out=grown)
        tables.resize(grown)
        tables.slot_map(lens, nodes, off, slots)
        spec.fp8_kv_append(*p.descs, kn, vn, slots)
        spec.fp8_tree_attention(q, *p.descs, tables.table, lens, off, mask, t, 8 * 16, out, 0.0, ws)
        spec.fp8_kv_accept(*p.descs, tables.table, lens, path, acc, lens)
        tables.resize(lens)

    graph = None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()                                     # nothing to do yet: no nodes, nothing accepted
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for _ in range(steps):
        trees = rng.integers(1, t + 1, b)
        sees = random_sees(rng, trees.tolist())
        n = int(trees.sum())
        x = rng.standard_normal((2, n, h, dim)).astype(np.float16)
        qq = rng.standard_normal((n, hq, dim)).astype(np.float16)
        paths = np.zeros((b, 4), np.int32)
        counts, start = np.zeros(b, np.int32), np.concatenate([[0], np.cumsum(trees)])
        for bi in range(b):
            leaf = int(rng.integers(trees[bi]))
            way = np.flatnonzero(sees[start[bi] + leaf])[:4]
            counts[bi] = int(rng.integers(0, len(way) + 1))
            paths[bi, : len(way)] = way
        for buf, val in ((q, qq), (kn, x[0]), (vn, x[1])):
            buf[:n].copy_(dev(val))
        mask[:n].copy_(spec.pack_tree_mask(dev(sees)))
        nodes.copy_(i32(trees))
        path.copy_(dev(paths))
        acc.copy_(dev(counts))
        step() if graph is None else graph.replay()
        got = host(out)
        for bi in range(b):
            # plain decode: each node after the accepted tokens and its own ancestors, in order
            for i in range(trees[bi]):
                way = start[bi] + np.flatnonzero(sees[start[bi] + i])
                seq = np.concatenate([tokens[bi], x[:, way]], 1).transpose(0, 2, 1, 3)[:, None]
                pools = [fp8.quantize(s, p.scale[r][0], fmt) for r, s in enumerate(seq)]
                for g in (0, hq - 1):
                    kk, vv = (fp8.decode(pools[r][0, g // gq], fmt) * np.float64(p.scale[r][0]) for r in range(2))
                    s = kk @ qq[start[bi] + i, g].astype(np.float64) / np.sqrt(dim)
                    w = np.exp(s - s.max())
                    ref = w @ vv / w.sum()
                    # scores within 1e-5 of exact at these sizes (tree_bound), values of unit size
                    assert np.abs(got[start[bi] + i, g] - ref).max() <= 1e-4
            keep = start[bi] + paths[bi, : counts[bi]]
            tokens[bi] = np.concatenate([tokens[bi], x[:, keep]], 1)
        assert host(lens).tolist() == [s.shape[1] for s in tokens]
        assert host(tables.n_held).tolist() == [-(-s.shape[1] // 16) for s in tokens]
        assert int(host(tables.free_count)[0]) == 40 - sum(-(-s.shape[1] // 16) for s in tokens)
    # the cache holds exactly the accepted tokens' bytes
    table = host(tables.table)
    for r, order in ((0, KEY), (1, VALUE)):
        nat = layout.fp8_unpack_pool(host(p.pool[r].view()), dim, order)
        for bi, s in enumerate(tokens):
            want = fp8.quantize(s[r].transpose(1, 0, 2)[None], p.scale[r][0], fmt)[0]
            for hi in range(h):
                assert np.array_equal(fp8.gather_paged(nat, table, bi, hi, s.shape[1]), want[hi])


def test_calls_on_another_stream():
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(31)
    p = Pools(rng, 8, 2, 64, "e4m3", False)
    x = rng.standard_normal((50, 2, 64)).astype(np.float16)
    dx, slots = dev(x), dev(np.arange(3, 53))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        spec.fp8_kv_append(*p.descs, dx, dx, slots)
    spec.fp8_kv_append(*p.descs, dx, dx, slots, stream=side)
    side.synchronize()
    for r in range(2):
        p.nat[r] = ospec.append(p.nat[r], x, np.arange(3, 53), p.scale[r][0], "e4m3")
    p.check()


def test_binding_checks_arguments():
    import torch
    kvq, spec = _mods()
    rng = np.random.default_rng(32)
    p = Pools(rng, 4, 2, 64, "e4m3", False)
    q = torch.zeros((3, 4, 64), dtype=torch.float16, device="cuda")
    table, lens, off = i32([[0, 1]]), i32([5]), i32([0, 3])
    mask = torch.zeros((3, 1), dtype=torch.int64, device="cuda")
    ws = spec.tree_workspace(1, 2, 4, 64, 3)
    out = torch.empty_like(q)

    def call(**kw):
        a = dict(q=q, k=p.descs[0], v=p.descs[1], table=table, lens=lens, off=off, mask=mask, max_tree=3, max_seq=32, out=out,
                 scale=0.0, ws=ws)
        a.update(kw)
        spec.fp8_tree_attention(*a.values())

    call()
    for bad in (dict(q=q.float()), dict(lens=lens.long()), dict(off=off[:1]), dict(mask=mask.int()), dict(out=out[:2]),
                dict(table=table.cpu()), dict(q=q.transpose(0, 1)), dict(out=out.double()), dict(mask=mask[:2]),
                dict(q=torch.zeros((3, 4, 128), dtype=torch.float16, device="cuda"))):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    with pytest.raises(kvq.KvqError):
        call(k=p.descs[1])
    with pytest.raises(kvq.KvqError):
        call(ws=ws[:0])
    with pytest.raises(ValueError):
        spec.fp8_kv_append(*p.descs, q[:, :2], q[:2, :2], dev(np.arange(3)))
    with pytest.raises(ValueError):
        spec.kv_blocks_resize(table, lens, i32([1, 2]), 16, i32([0]), i32([0]))
