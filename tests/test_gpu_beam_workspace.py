"""One workspace of the block calls for pools of several sizes and any number of requests."""
import numpy as np
import pytest

from oracle import beam as obeam
from kvq_helpers import dev, host
from test_gpu_beam import State, empty, i32, random_tables

pytestmark = pytest.mark.gpu


def compact(ws, rng, blocks, keep):
    """Compacts random tables over a pool of this size, and compares them with the oracle's."""
    from quantized_kv_cache_quant_gb300 import beam
    table, held, shares, free = random_tables(rng, 8, 60, blocks, 40)
    stack = np.full(blocks, -7, np.int32)
    stack[: len(free)] = free
    d = dict(table=dev(table), held=dev(held), shares=dev(shares), free=dev(stack), count=i32([len(free)]), moved=empty((blocks,)),
             src=empty((blocks,)), dst=empty((blocks,)), n=empty((1,)), done=empty((1,)))
    beam.kv_blocks_compact(d["table"], d["held"], keep, d["shares"], d["free"], d["count"], d["moved"], d["src"], d["dst"],
                           d["n"], d["done"], ws)
    r = obeam.compact(table, held, keep, shares, free, blocks)
    assert host(d["done"])[0] == r["done"] and np.array_equal(host(d["table"]), r["table"])
    assert host(d["moved"]).tolist() == r["moved_to"] and np.array_equal(host(d["shares"]), r["shares"])
    assert host(d["free"])[: host(d["count"])[0]].tolist() == list(r["free"])


@pytest.mark.parametrize("sizes", [(400, 3000), (3000, 400), (700, 40000), (20000, 90000), (90000, 700)])
def test_pools_of_other_sizes_share_a_workspace(sizes):
    from quantized_kv_cache_quant_gb300 import beam
    rng = np.random.default_rng(sizes[0])
    ws = beam.blocks_workspace(50, 100000)
    assert ws.numel() >= beam.kv_blocks_workspace_bytes(50, max(sizes) + 9000)
    for requests, width in ((3, 4), (50, 2), (1, 8)):
        for blocks in sizes:
            compact(ws, rng, blocks, blocks - blocks // 8)
            s = State(rng, requests, width, 40, 16, 0)
            s.free = []
            spare = blocks - s.blocks
            if spare > 0:                                 # (a pool of the asked size, with that many free blocks)
                s.shares = np.concatenate([s.shares, np.zeros(spare, np.int32)])
                s.free = rng.permutation(np.arange(s.blocks, blocks)).tolist()
                s.blocks = blocks
                s._push()
            s.ws = ws
            s.d["free"].fill_(-7)
            s.d["free"][: len(s.free)] = i32(s.free)
            s.d["count"].fill_(len(s.free))
            from_parents(s, rng, requests, width)


def from_parents(s, rng, requests, width):
    from quantized_kv_cache_quant_gb300 import beam
    d, parents = s.d, rng.integers(-1, width, requests * width)
    beam.kv_blocks_fork(d["table"], d["held"], d["lens"], i32(parents), width, 16, d["shares"], d["free"], d["count"], d["src"],
                        d["dst"], d["n"], s.ws, d["granted"], d["shared"])
    r = obeam.fork(s.table, s.held, s.lens, parents, width, 16, s.shares, s.free)
    g = {k: host(v) for k, v in d.items()}
    assert np.array_equal(g["table"], r["table"]) and np.array_equal(g["shares"], r["shares"])
    assert g["count"][0] == len(r["free"]) and g["free"][: len(r["free"])].tolist() == list(r["free"])
    assert g["granted"].tolist() == r["granted"] and g["shared"].tolist() == r["shared"]
