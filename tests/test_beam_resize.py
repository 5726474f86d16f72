"""Tables that share blocks: a resize gives up no block that others hold, and how such a sequence is shortened."""
import numpy as np
import pytest

from oracle import spec as ospec

kvq = pytest.importorskip("quantized_kv_cache_quant_gb300.kvq", reason="libkvq.so not built")
beam = pytest.importorskip("quantized_kv_cache_quant_gb300.beam")

A = 1 << 20  # a fake, 256-byte aligned address: the checks never read through it
NULL, ARG, UNSUPPORTED, ALIGN = 1, 2, 6, 9
ARGS = dict(table=A, batch=8, max_blocks=10, held=A, target=A, bt=16, shares=A, free=A, count=A, blocks=64, granted=None,
            stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, NULL) for k in ("table", "held", "target", "shares", "free", "count")],
    (dict(batch=0), ARG), (dict(max_blocks=0), ARG), (dict(bt=0), ARG), (dict(blocks=0), ARG), (dict(batch=4097), UNSUPPORTED),
    (dict(max_blocks=1 << 29), UNSUPPORTED), (dict(table=A + 4), ALIGN), (dict(shares=A + 4), ALIGN),
    (dict(granted=A + 4), ALIGN), (dict(target=A + 4), ALIGN)])
def test_refusals(change, code):
    assert kvq._lib.kv_blocks_resize_shared(*dict(ARGS, **change).values()) == code


def i32(x):
    from kvq_helpers import dev
    return dev(np.asarray(x, np.int32))


@pytest.mark.gpu
def test_a_shrink_of_shared_blocks_is_refused():
    from kvq_helpers import host
    t = beam.BeamTables(1, 3, 8, 20)
    t.resize(i32([50, 0, 0]))
    t.seq_lens.copy_(i32([50, 0, 0]))
    t.fork(i32([0, 0, 0]))                                # 3 full blocks shared, 3 last ones of their own
    before = host(t.table).copy()
    t.resize(i32([16, 60, 90]))                           # the first would give up blocks of the others
    assert host(t.granted).tolist() == [0, 1, 1] and host(t.n_held).tolist() == [4, 4, 6]
    after = host(t.table)
    assert np.array_equal(after[:2], before[:2]) and np.array_equal(after[2, :4], before[2, :4])
    t.resize(i32([48, 48, 48]))                           # blocks of their own
    assert host(t.granted).tolist() == [1, 1, 1] and host(t.n_held).tolist() == [3, 3, 3]
    assert int(host(t.free_count)[0]) == 17
    t.resize(i32([0, 0, 0]))
    assert host(t.granted).tolist() == [0, 0, 0] and int(host(t.free_count)[0]) == 17


@pytest.mark.gpu
@pytest.mark.parametrize("requests,width,max_blocks,bt,spare", [
    (1, 1, 4, 16, 8), (3, 4, 9, 16, 30), (40, 8, 70, 16, 500), (1000, 4, 9, 1, 3000), (5, 3, 6000, 16, 200)])
def test_resize_of_shared_tables_matches_oracle(requests, width, max_blocks, bt, spare):
    from kvq_helpers import dev, host
    from test_gpu_beam import State
    rng = np.random.default_rng(requests + max_blocks)
    s = State(rng, requests, width, max_blocks, bt, spare, pinned=min(3, requests - 1))
    d, b = s.d, requests * width
    table, held, free = s.table, s.held, list(s.free)
    for step in range(3):
        target = np.maximum(0, held * bt + rng.integers(-3 * bt, 2 * bt, b))
        if step == 1:
            target[rng.random(b) < 0.3] = 0
        beam.kv_blocks_resize_shared(d["table"], d["held"], dev(target.astype(np.int32)), bt, d["shares"], d["free"], d["count"],
                                     d["granted"])
        want = target.copy()
        for i in range(b):
            if target[i] > max_blocks * bt or (s.shares[table[i, -(-target[i] // bt): held[i]]] > 0).any():
                want[i] = -1
        table, held, free, ok = ospec.resize(table, held, want, bt, free)
        assert np.array_equal(host(d["table"]), table) and np.array_equal(host(d["held"]), held)
        assert host(d["count"])[0] == len(free) and host(d["free"])[: len(free)].tolist() == list(free)
        assert np.array_equal(host(d["granted"]), ok) and np.array_equal(host(d["shares"]), s.shares)


@pytest.mark.gpu
@pytest.mark.parametrize("requests,width,max_blocks", [(1, 4, 7), (5, 5, 33), (64, 8, 130), (1024, 4, 9)])
def test_sequences_are_shortened_by_a_fork_to_themselves(requests, width, max_blocks):
    """Lower lengths, every sequence its own parent: blocks that nobody holds any more come back, and a block that is full
    for others and partly filled now is copied."""
    from kvq_helpers import dev
    from test_gpu_beam import State
    rng = np.random.default_rng(requests)
    s = State(rng, requests, width, max_blocks, 16, 4 * requests * width)
    own = np.tile(np.arange(width), requests)
    for _ in range(3):
        s.lens = rng.integers(0, s.lens + 1).astype(np.int32)
        s.d["lens"].copy_(dev(s.lens))
        s.fork(own)
