"""Beam search over the paged caches on the GPU: candidates, tables, copies and
compaction equal the oracle's."""
import numpy as np
import pytest

from oracle import beam as obeam
from kvq_helpers import dev, host

pytestmark = pytest.mark.gpu


def _mods():
    from quantized_kv_cache_quant_gb300 import beam, kvq
    return beam, kvq


def i32(x):
    return dev(np.asarray(x, np.int32))


def empty(shape, kind="int32"):
    import torch
    return torch.full(shape, -7, dtype=getattr(torch, kind), device="cuda")


# ---------------------------------------------------------------- selection

def run_select(x, scores, n, finished=None, end=-1):
    beam, _ = _mods()
    r = scores.shape[0]
    out = empty((r, n), "float32"), empty((r, n)), empty((r, n))
    beam.beam_select(x, dev(scores), *out, None if finished is None else dev(finished), end)
    return [host(o) for o in out]


def check_select(x, scores, n, finished=None, end=-1, got=None):
    """x: a device tensor [R * W, V]. Scores within what the arithmetic allows: an exponential is off by 2 ulp and its
    argument's rounding (2^-24 |d| e^d <= 2^-25.4), a thread's sum adds at most 2^-24 a term, of which there are up to V /
    512 + 32 in one after the other, the output's rounding 2^-24 of its size. Candidates have to be the oracle's but
    where two scores are closer than twice that."""
    s, p, t = run_select(x, scores, n, finished, end) if got is None else got
    xs = host(x.float())
    want, wp, wt = obeam.select(xs, scores, n, finished, end)
    v = xs.shape[1]
    assert ((t >= 0) & (t < v)).all() and ((p >= 0) & (p < scores.shape[1])).all()
    fin = np.isfinite(want)
    tol = 2.0**-24 * (np.abs(np.where(fin, want, 0.0)) + 16 + v / 512 + 32)
    assert np.array_equal(fin, np.isfinite(s)) and (s[~fin] == -np.inf).all()
    assert (np.abs(np.where(fin, s, 0) - np.where(fin, want, 0)) <= tol).all()
    for g in range(len(s)):
        assert len({(a, b) for a, b in zip(p[g], t[g])}) == n
        for i in np.flatnonzero((p[g] != wp[g]) | (t[g] != wt[g])):
            gaps = [abs(want[g, i] - want[g, j]) for j in range(n) if j != i and fin[g, i] and fin[g, j]]
            # (the last one may be as close to the first candidate left out)
            assert fin[g, i] and (i == n - 1 or min(gaps) <= 2 * tol[g, i]), (g, i, p[g], t[g], wp[g], wt[g])


TYPES = ["float16", "float32", "bfloat16"]


def logits(rng, rows, v, kind, spread=2.0):
    import torch
    x = rng.standard_normal((rows, v)).astype(np.float32) * spread
    x[:, : 20] += 5
    x = rng.permuted(x, axis=1)
    return dev(x).to(getattr(torch, kind))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("r,w,v,n", [
    (1, 1, 1, 1), (1, 2, 3, 3), (2, 3, 17, 5), (1, 4, 32000, 4), (3, 5, 999, 10), (7, 1, 50021, 1), (2, 8, 4097, 16),
    (1, 64, 300, 128), (40, 4, 2048, 8), (300, 2, 777, 4), (1, 3, 131072, 128), (5, 16, 16385, 32)])
def test_select_matches_oracle(r, w, v, n, kind):
    rng = np.random.default_rng(r * 1000 + w * 100 + v)
    x = logits(rng, r * w, v, kind)
    check_select(x, rng.uniform(-20, 0, (r, w)).astype(np.float32), n)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("shift,gap", [(1, 1), (3, 5), (0, 8), (7, 3)])
def test_select_rows_that_start_anywhere(shift, gap, kind):
    import torch
    rng = np.random.default_rng(shift)
    whole = torch.full((6, 1000 + shift + gap), float("nan"), dtype=getattr(torch, kind), device="cuda")
    whole[:, shift:shift + 1000] = logits(rng, 6, 1000, kind)
    check_select(whole[:, shift:shift + 1000], rng.uniform(-9, 0, (2, 3)).astype(np.float32), 7)


@pytest.mark.parametrize("kind", TYPES)
def test_select_with_ended_and_dead_beams(kind):
    rng = np.random.default_rng(5)
    x = logits(rng, 24, 3001, kind)
    finished = rng.random((6, 4)) < 0.4
    finished[2] = True
    scores = rng.uniform(-9, -3, (6, 4)).astype(np.float32)
    scores[1, 2], scores[3, 0], scores[4, 1] = -np.inf, np.nan, np.inf
    scores[5] = -np.inf
    finished[1, 2], finished[3, 0], finished[4, 1] = False, True, False
    finished[5] = [False, True, False, True]
    for end in (0, 1, 1234, 3000):
        check_select(x, scores, 9, finished, end)
        check_select(x, scores, 9, finished.astype(np.uint8), end)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("left", [0, 1, 3, 40])
def test_select_where_bans_leave_few_tokens(kind, left):
    """Rows that keep `left` tokens: candidates at -inf fill up by their index; NaN counts as banned."""
    rng = np.random.default_rng(left)
    x = logits(rng, 6, 40000, kind)
    for row in range(6):
        keep = rng.permutation(40000)[:left]
        banned = np.ones(40000, bool)
        banned[keep] = False
        x[row, dev(banned)] = float("nan") if row % 2 else -float("inf")
    check_select(x, rng.uniform(-9, -3, (2, 3)).astype(np.float32), 12)


@pytest.mark.parametrize("kind", TYPES)
def test_select_infinities_and_signed_zeros(kind):
    import torch
    x = torch.zeros((4, 500), dtype=getattr(torch, kind), device="cuda")
    x[0, ::2] = -0.0                                     # equal values: the lowest tokens
    x[1, 300] = x[1, 7] = float("inf")
    x[2] = float("-inf")
    x[3] = torch.finfo(x.dtype).min
    big = float(np.finfo(np.float32).max)
    y = x.float().clamp(max=big)
    s, p, t = run_select(x, np.zeros((4, 1), np.float32), 5)
    want = obeam.select(host(y), np.zeros((4, 1), np.float32), 5)
    assert np.array_equal(t, want[2]) and np.allclose(s, want[0], atol=1e-5)


@pytest.mark.parametrize("at", [-65536.0, -1e6, 30000.0, 65000.0, 65536.0, 1e6, 1e30, 3e38])
def test_select_of_large_logits(at):
    """Rows far from zero, as a whole and from their middle on: a difference of logits stays exact."""
    rng = np.random.default_rng(11)
    x = rng.integers(-8, 8, (6, 30000)).astype(np.float32)
    x[:3] += np.float32(at)
    x[3:, 15000:] += np.float32(at)
    check_select(dev(x), rng.uniform(-9, 0, (2, 3)).astype(np.float32), 5)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("order", ["equal", "rising", "falling", "steps"])
def test_select_of_rows_that_fill_the_lists(kind, order):
    """Every element reaches the bound, or every chunk exceeds what came before it."""
    import torch
    v = 70000
    i = torch.arange(v, device="cuda", dtype=torch.float32)
    x = {"equal": 0 * i, "rising": i / v * 20, "falling": -i / v * 20, "steps": (i // 9000)}[order]
    x = x.to(getattr(torch, kind)).repeat(4, 1)
    for n in (1, 16, 128):
        check_select(x, np.array([[0, -1.5], [-2.25, -2.25]], np.float32), n)


def test_select_equal_beams_go_to_the_lower_one():
    rng = np.random.default_rng(8)
    x = logits(rng, 1, 5003, "float32").repeat(12, 1)     # rows start at other boundaries of 16 bytes
    s, p, t = run_select(x, np.zeros((3, 4), np.float32), 8)
    for g in range(3):
        assert p[g].tolist() == [0, 1, 2, 3] * 2 and len(set(t[g][:4])) == 1 and len(set(t[g][4:])) == 1


def test_select_is_the_same_every_time():
    rng = np.random.default_rng(9)
    x = logits(rng, 512, 20000, "bfloat16")
    scores = rng.uniform(-9, 0, (64, 8)).astype(np.float32)
    first = run_select(x, scores, 16)
    for _ in range(20):
        for a, b in zip(first, run_select(x, scores, 16)):
            assert np.array_equal(a, b)


def test_select_of_many_elements():
    """Offsets beyond 31 bits, requests of one row."""
    import torch
    v, rows = 140000, 16000
    x = torch.randn((rows, v), dtype=torch.float16, device="cuda")
    r = torch.arange(rows, device="cuda")
    x[r, (r * 7919) % v] = 20.0
    out = empty((rows, 1), "float32"), empty((rows, 1)), empty((rows, 1))
    beam, _ = _mods()
    beam.beam_select(x, torch.zeros((rows, 1), device="cuda"), *out)
    assert torch.equal(out[2][:, 0], ((r * 7919) % v).int()) and int(out[1].abs().max()) == 0


def test_select_on_two_streams_and_captured():
    import torch
    beam, _ = _mods()
    rng = np.random.default_rng(10)
    x = [logits(rng, 20, 30011, "float16") for _ in range(2)]
    scores = [dev(rng.uniform(-9, 0, (5, 4)).astype(np.float32)) for _ in range(2)]
    out = [(empty((5, 8), "float32"), empty((5, 8)), empty((5, 8))) for _ in range(2)]
    want = []
    for i in range(2):
        beam.beam_select(x[i], scores[i], *out[i])
        torch.cuda.synchronize()
        want.append([o.clone() for o in out[i]])
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        streams[i].wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i], stream=streams[i]):
            beam.beam_select(x[i], scores[i], *out[i])
    for how in ("eager", "argument", "graph"):
        for o in out[0] + out[1]:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            for i in range(2):
                if how == "argument":
                    beam.beam_select(x[i], scores[i], *out[i], stream=streams[i])
                    continue
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay() if how == "graph" else beam.beam_select(x[i], scores[i], *out[i])
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in zip(out[i], want[i]):
                assert torch.equal(a, b)


# ---------------------------------------------------------------- fork

class State:
    """Random tables of requests whose sequences share leading blocks, on the host and on the device."""

    def __init__(self, rng, requests, width, max_blocks, bt, spare, pinned=0):
        self.width, self.bt = width, bt
        b = requests * width
        rows, lens = [], []
        n = 0
        for g in range(requests):
            lead = int(rng.integers(0, max_blocks))
            for i in range(width):
                own = int(rng.integers(0, min(4, max_blocks - lead) + 1))
                empty_row = rng.random() < 0.15 or lead + own == 0
                rows.append(None if empty_row else (g, lead, own))
                lens.append(0 if empty_row else int(rng.integers((lead + own - 1) * bt + 1, (lead + own) * bt + 1)))
        total = requests * max_blocks + 4 * b + spare
        perm = rng.permutation(total)
        lead_blocks = {g: perm[g * max_blocks:(g + 1) * max_blocks] for g in range(requests)}
        n = requests * max_blocks
        self.table = np.full((b, max_blocks), -1, np.int32)
        self.held = np.zeros(b, np.int32)
        refs = np.zeros(total, np.int64)
        for i, row in enumerate(rows):
            if row is None:
                continue
            g, lead, own = row
            self.table[i, :lead] = lead_blocks[g][:lead]
            self.table[i, lead:lead + own] = perm[n:n + own]
            n += own
            self.held[i] = lead + own
            refs[self.table[i, : lead + own]] += 1
        self.lens = np.array(lens, np.int32)
        # a partly filled last block that several share is allowed: lead blocks with own = 0
        used = refs > 0
        self.shares = np.maximum(refs - 1, 0).astype(np.int32)
        if pinned:                                        # references from outside the tables
            at = rng.permutation(np.flatnonzero(used))[:pinned]
            self.shares[at] += 1
        self.free = rng.permutation(np.flatnonzero(~used)).tolist()[:max(0, spare)] if spare < total else []
        self.blocks = total
        self._push()

    def _push(self):
        stack = np.full(self.blocks, -7, np.int32)
        stack[: len(self.free)] = self.free
        b = len(self.held)
        self.d = dict(table=dev(self.table), held=dev(self.held), lens=dev(self.lens), shares=dev(self.shares), free=dev(stack),
                      count=i32([len(self.free)]), src=empty((b,)), dst=empty((b,)), n=empty((1,)), granted=empty((b,)),
                      shared=empty((b // self.width,)))
        beam, _ = _mods()
        self.ws = beam.blocks_workspace(max(1, b // self.width), self.blocks)

    def fork(self, parents, optional=True):
        beam, _ = _mods()
        d = self.d
        beam.kv_blocks_fork(d["table"], d["held"], d["lens"], i32(parents), self.width, self.bt, d["shares"], d["free"],
                            d["count"], d["src"], d["dst"], d["n"], self.ws, d["granted"] if optional else None,
                            d["shared"] if optional else None)
        r = obeam.fork(self.table, self.held, self.lens, parents, self.width, self.bt, self.shares, self.free)
        self.check(r, optional)
        return r

    def check(self, r, optional=True):
        d = {k: host(v) for k, v in self.d.items()}
        self.table, self.shares, self.free = np.array(r["table"], np.int32), np.array(r["shares"], np.int32), r["free"]
        self.held, self.lens = np.array(r["held"], np.int32), np.array(r["lens"], np.int32)
        assert np.array_equal(d["table"], self.table)
        assert np.array_equal(d["held"], self.held) and np.array_equal(d["lens"], self.lens)
        assert d["count"][0] == len(self.free) and d["free"][: len(self.free)].tolist() == list(self.free)
        assert np.array_equal(d["shares"], self.shares)
        assert d["n"][0] == len(r["pairs"])
        assert list(zip(d["src"].tolist(), d["dst"].tolist()))[: len(r["pairs"])] == [tuple(map(int, p)) for p in r["pairs"]]
        if optional:
            assert d["granted"].tolist() == r["granted"] and d["shared"].tolist() == r["shared"]
        # the calls leave their workspace as they need it
        assert int(self.ws[256:].max()) == 0


@pytest.mark.parametrize("requests,width,max_blocks,bt,spare,pinned", [
    (1, 1, 1, 16, 3, 0), (1, 4, 7, 16, 10, 0), (3, 4, 5, 1, 30, 3), (8, 4, 70, 16, 40, 10), (5, 5, 33, 32, 0, 0),
    (2, 64, 40, 16, 200, 20), (64, 8, 130, 16, 300, 40), (600, 1, 20, 16, 50, 0), (1024, 4, 9, 16, 2000, 100),
    (1, 3, 5000, 16, 4, 0), (20, 7, 300, 16, 3, 5)])
def test_fork_matches_oracle(requests, width, max_blocks, bt, spare, pinned):
    rng = np.random.default_rng(requests * 7 + width)
    s = State(rng, requests, width, max_blocks, bt, spare, pinned)
    b = requests * width
    for step in range(5):
        parents = rng.integers(-1, width + 1, b)          # some out of range: those sequences end
        if step == 1:
            parents = np.tile(np.arange(width), requests)  # every one itself
        if step == 3:
            parents = np.zeros(b, int)                    # all from the first
        s.fork(parents, optional=step != 2)


def test_fork_of_a_large_pool():
    """Words of more than one thread block, blocks freed all over them."""
    rng = np.random.default_rng(3)
    s = State(rng, 40, 4, 600, 16, 400000)
    s.fork(rng.integers(0, 4, 160))
    s.fork(np.full(160, -1))                              # everything comes back
    assert (s.table == -1).all() and s.shares.sum() == 0


def test_fork_with_a_state_that_does_not_add_up_stays_inside():
    import torch
    beam, _ = _mods()
    table = dev(np.array([[3, 3, 99, -5], [3, 2, 1, 0], [2**31 - 1, 0, 0, 0], [1, 1, 1, 1]], np.int32))
    held, lens = i32([99, 4, -3, 4]), i32([2**31 - 1, 50, 7, 64])
    free, count, shares = i32([7, 7, 7, -9]), i32([77]), i32([0, 0, 0, 0])
    ws = beam.blocks_workspace(1, 4)
    src, dst, n = empty((4,)), empty((4,)), empty((1,))
    for parents in ([1, 0, 3, 2], [0, 0, 0, 0], [-1] * 4):
        beam.kv_blocks_fork(table, held, lens, i32(parents), 4, 16, shares, free, count, src, dst, n, ws)
    torch.cuda.synchronize()
    assert host(held).tolist() == [0] * 4 and host(lens).tolist() == [0] * 4 and 0 <= host(count)[0] <= 4


def test_fork_captured_and_replayed_with_new_parents():
    import torch
    rng = np.random.default_rng(12)
    s = State(rng, 6, 4, 30, 16, 60)
    beam, _ = _mods()
    d, parents = s.d, i32(np.tile(np.arange(4), 6))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    saved = {k: v.clone() for k, v in d.items()}
    with torch.cuda.graph(graph, stream=side):
        beam.kv_blocks_fork(d["table"], d["held"], d["lens"], parents, 4, 16, d["shares"], d["free"], d["count"], d["src"],
                            d["dst"], d["n"], s.ws, d["granted"], d["shared"])
    for k, v in saved.items():
        assert torch.equal(d[k], v)                       # nothing ran yet
    for _ in range(4):
        p = rng.integers(0, 4, 24)
        parents.copy_(i32(p))
        graph.replay()
        s.check(obeam.fork(s.table, s.held, s.lens, p, 4, 16, s.shares, s.free))


# ---------------------------------------------------------------- copies

@pytest.mark.parametrize("sizes,blocks,pairs,used", [
    ([16], 2, 1, None), ([64, 4096, 4112], 40, 15, None), ([16384] * 5, 100, 40, 7), ([9 * 128 * 2] * 3 + [2048], 60, 30, 0),
    ([1024] * 160, 50, 25, 25), ([100000], 64, 32, 99), ([3 * 16], 9000, 4000, 3777)])
def test_copy_moves_whole_blocks(sizes, blocks, pairs, used):
    import torch
    beam, _ = _mods()
    rng = np.random.default_rng(blocks)
    bufs = [torch.randint(0, 256, (blocks, n), dtype=torch.uint8, device="cuda") for n in sizes]
    was = [host(b).copy() for b in bufs]
    perm = rng.permutation(blocks)
    src, dst = perm[rng.integers(0, pairs, pairs)], perm[pairs:2 * pairs]
    count = None if used is None else i32([used])
    beam.kv_blocks_copy(beam.BlockBuffers(blocks, bufs), i32(src), i32(dst), count)
    n = pairs if used is None else min(used, pairs)
    for b, w in zip(bufs, was):
        w[dst[:n]] = w[src[:n]]
        assert np.array_equal(host(b), w)


def test_copy_skips_pairs_outside_the_pool():
    import torch
    beam, _ = _mods()
    buf = torch.arange(8, device="cuda", dtype=torch.uint8)[:, None].repeat(1, 256)
    beam.kv_blocks_copy(beam.BlockBuffers(8, [buf]), i32([-1, 8, 2, 3, 2**31 - 1]), i32([0, 1, 8, -2, 4]))
    assert host(buf)[:, 0].tolist() == list(range(8))
    beam.kv_blocks_copy(beam.BlockBuffers(8, [buf]), i32([1]), i32([0]), i32([-5]))
    assert host(buf)[:, 0].tolist() == list(range(8))


def test_copy_captured_follows_the_count():
    import torch
    beam, _ = _mods()
    buf = torch.arange(40, device="cuda", dtype=torch.uint8)[:, None].repeat(1, 4096)
    bufs, count = beam.BlockBuffers(40, [buf]), i32([0])
    src, dst = i32(range(20)), i32(range(20, 40))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        beam.kv_blocks_copy(bufs, src, dst, count)
    for n in (0, 1, 7, 20):
        count.fill_(n)
        graph.replay()
        want = list(range(20)) + [i if i < n else 20 + i for i in range(20)]
        assert host(buf).min(1).tolist() == host(buf).max(1).tolist() == want


@pytest.mark.parametrize("dim", [64, 128])
def test_copied_blocks_of_the_other_pools_decode_alike(dim):
    """NVFP4 pools: a sequence whose blocks are copies of another's decodes to the same bits."""
    import torch
    beam, kvq = _mods()
    rng = np.random.default_rng(dim)
    x = rng.standard_normal((2, 1, 2, 64, dim)).astype(np.float16)
    pools = [kvq.Nvfp4Pool(role, 8, 2, dim) for role in (kvq.ROLE_KEY, kvq.ROLE_VALUE)]
    for p, y in zip(pools, x):
        p.quantize(dev(y), i32([[0, 1, 2, 3]]), 4)
    beam.kv_blocks_copy(beam.BlockBuffers(8, [p.view() for p in pools]), i32([0, 1, 2, 3]), i32([7, 5, 4, 6]))
    q = dev(np.repeat(rng.standard_normal((1, 8, dim)).astype(np.float16), 2, 0))
    out = torch.empty((2, 8, dim), dtype=torch.float32, device="cuda")
    n = kvq.nvfp4_decode_workspace_bytes(2, 8, dim)
    kvq.nvfp4_decode_attention(q, *(p.desc for p in pools), i32([[0, 1, 2, 3], [7, 5, 4, 6]]), i32([60, 60]), 2, 8, 4, 64, out,
                               True, 0.0, torch.zeros(n, dtype=torch.uint8, device="cuda"), n)
    assert torch.equal(out[0], out[1]) and float(out.abs().max()) > 0


def test_copy_beyond_31_bits():
    import torch
    beam, _ = _mods()
    size, blocks = 1 << 20, 5000
    buf = torch.zeros((blocks, size), dtype=torch.uint8, device="cuda")
    buf[4999], buf[2500] = 5, 9
    beam.kv_blocks_copy(beam.BlockBuffers(blocks, [buf]), i32([4999, 2500]), i32([3, 4998]))
    assert int(buf[3].min()) == int(buf[3].max()) == 5 and int(buf[4998].min()) == int(buf[4998].max()) == 9
    assert int(buf[2].max()) == 0 and int(buf[4997].max()) == 0


# ---------------------------------------------------------------- compaction

def random_tables(rng, batch, width, blocks, most):
    held = rng.integers(0, most + 1, batch)
    perm = rng.permutation(blocks)
    table, at = np.full((batch, width), -1, np.int32), 0
    shares = np.zeros(blocks, np.int32)
    for b, n in enumerate(held):
        n = min(int(n), width, blocks - at)
        held[b] = n
        table[b, :n] = perm[at:at + n]
        at += n
        if b and n and held[b - 1]:                       # some blocks are shared with the row before
            table[b, 0] = table[b - 1, 0]
    for x, c in zip(*np.unique(table[table >= 0], return_counts=True)):
        shares[x] = c - 1
    used = set(table[table >= 0].tolist())
    outside = {int(x) for x in perm[at:at + max(0, (blocks - at) // 10)]}   # held by nobody in the tables
    free = [int(x) for x in rng.permutation(blocks) if x not in used and x not in outside]
    return table, held.astype(np.int32), shares, free


def run_compact(table, held, keep, shares, free, room):
    beam, _ = _mods()
    blocks = len(shares)
    stack = np.full(blocks, -7, np.int32)
    stack[: len(free)] = free
    d = dict(table=dev(table), held=dev(held), shares=dev(shares), free=dev(stack), count=i32([len(free)]), moved=empty((blocks,)),
             src=empty((room,)), dst=empty((room,)), n=empty((1,)), done=empty((1,)))
    ws = beam.blocks_workspace(1, blocks)
    beam.kv_blocks_compact(d["table"], d["held"], keep, d["shares"], d["free"], d["count"], d["moved"], d["src"], d["dst"],
                           d["n"], d["done"], ws)
    r = obeam.compact(table, held, keep, shares, free, room)
    g = {k: host(v) for k, v in d.items()}
    assert g["done"][0] == r["done"]
    assert np.array_equal(g["table"], r["table"]) and np.array_equal(g["shares"], r["shares"])
    assert g["count"][0] == len(r["free"]) and g["free"][: len(r["free"])].tolist() == list(r["free"])
    assert g["moved"].tolist() == r["moved_to"] and g["n"][0] == len(r["pairs"])
    assert list(zip(g["src"].tolist(), g["dst"].tolist()))[: len(r["pairs"])] == r["pairs"]
    return r


@pytest.mark.parametrize("batch,width,blocks,most,keep", [
    (1, 1, 1, 1, 1), (1, 1, 1, 1, 0), (3, 5, 40, 4, 16), (3, 5, 40, 4, 17), (8, 100, 2000, 60, 900), (8, 100, 2000, 60, 0),
    (8, 100, 2000, 60, 2000), (40, 70, 9000, 60, 5000), (300, 1000, 300000, 500, 150001), (4096, 3, 20000, 3, 13000),
    (2, 9000, 20000, 8000, 17000)])
def test_compact_matches_oracle(batch, width, blocks, most, keep):
    rng = np.random.default_rng(batch + blocks)
    table, held, shares, free = random_tables(rng, batch, width, blocks, most)
    run_compact(table, held, keep, shares, free, max(1, blocks))


def test_compact_refuses_what_does_not_fit():
    rng = np.random.default_rng(4)
    table, held, shares, free = random_tables(rng, 8, 100, 700, 60)
    assert run_compact(table, held, 100, shares, free, 700)["done"] == 0      # too few free blocks below
    assert run_compact(table, held, 600, shares, free, 700)["done"] == 1
    assert run_compact(table, held, 600, shares, free, 1)["done"] == 0        # too small a list


# ---------------------------------------------------------------- refusals of the binding

def test_binding_checks_arguments():
    import torch
    beam, _ = _mods()
    x = torch.zeros((6, 50), device="cuda")
    s = torch.zeros((2, 3), device="cuda")
    o, p, t = empty((2, 4), "float32"), empty((2, 4)), empty((2, 4))
    beam.beam_select(x, s, o, p, t)
    for bad in (dict(x=x.double()), dict(x=x[:5]), dict(x=x.t()), dict(s=s.view(6)), dict(s=s.half()), dict(p=p[:1]),
                dict(t=t.long()), dict(o=o.t().contiguous().t())):
        a = dict(x=x, s=s, o=o, p=p, t=t, **{})
        a.update(bad)
        with pytest.raises((TypeError, ValueError)):
            beam.beam_select(*a.values())
    from quantized_kv_cache_quant_gb300 import kvq
    with pytest.raises(kvq.KvqError):
        beam.beam_select(x, s, empty((2, 51), "float32"), empty((2, 51)), empty((2, 51)))
    buf = beam.BlockBuffers(4, [torch.zeros((4, 64), device="cuda")])
    with pytest.raises(TypeError):
        beam.kv_blocks_copy(buf, torch.zeros(2, dtype=torch.int64, device="cuda"), i32([1, 2]))
    with pytest.raises(ValueError):
        beam.kv_blocks_copy(buf, i32([1, 2]), i32([1]))
    with pytest.raises(ValueError):
        beam.BlockBuffers(4, [torch.zeros((4, 64), device="cuda").t()])
