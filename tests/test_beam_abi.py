"""The beam-search calls without a GPU: exported symbols, limits, refusals (no
kernel is launched) and the oracle's tables."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import beam as obeam

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kvq_beam.h")

kvq = pytest.importorskip("quantized_kv_cache_quant_gb300.kvq", reason="libkvq.so not built")
beam = pytest.importorskip("quantized_kv_cache_quant_gb300.beam")

A = 1 << 20  # a fake, 256-byte aligned address: the checks never read through it
OK, NULL, ARG, SHAPE, CAPACITY, WORKSPACE, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4, 5, 6, 9


def test_declared_symbols_are_exported_and_bound():
    names = re.findall(r"KVQ_API\s+[\w\s\*]+?\b(\w+)\s*\(", open(HEADER, encoding="utf-8").read())
    assert sorted(names) == sorted(beam.EXPORTED) == sorted(beam._SIG)
    lib = ctypes.CDLL(kvq.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_limits_match_the_header():
    text = open(HEADER, encoding="utf-8").read()
    for name, value in (("KVQ_BEAM_MAX_WIDTH", beam.MAX_WIDTH), ("KVQ_BEAM_MAX_OUT", beam.MAX_OUT),
                        ("KVQ_COPY_MAX_BUFFERS", beam.COPY_MAX_BUFFERS)):
        assert int(re.search(rf"#define {name}\s+(\d+)", text).group(1)) == value


def _call(name, args, change):
    args = dict(args, **change)
    return getattr(kvq._lib, name)(*args.values())


SELECT = dict(logits=A, type=0, stride=1000, scores=A, finished=None, end=-1, groups=2, width=4, vocab=1000, n=8, os=A, op=A,
              ot=A, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), NULL), (dict(scores=None), NULL), (dict(os=None), NULL), (dict(op=None), NULL), (dict(ot=None), NULL),
    (dict(type=3), ARG), (dict(type=-1), ARG), (dict(groups=0), ARG), (dict(width=0), ARG), (dict(vocab=0), ARG),
    (dict(n=0), ARG), (dict(n=1001), ARG), (dict(stride=999), ARG), (dict(finished=A, end=-1), ARG),
    (dict(finished=A, end=1000), ARG), (dict(width=65), UNSUPPORTED), (dict(n=129), UNSUPPORTED),
    (dict(vocab=(1 << 30) + 1, stride=1 << 31), UNSUPPORTED), (dict(groups=(1 << 24) + 1), UNSUPPORTED),
    (dict(logits=A + 1), ALIGN), (dict(logits=A + 2, type=1), ALIGN), (dict(scores=A + 4), ALIGN), (dict(os=A + 4), ALIGN),
    (dict(op=A + 4), ALIGN), (dict(ot=A + 4), ALIGN), (dict(finished=A + 1, end=0), ALIGN)])
def test_select_refusals(change, code):
    assert _call("beam_select", SELECT, change) == code


FORK = dict(table=A, batch=8, max_blocks=10, held=A, lens=A, parents=A, width=4, bt=16, shares=A, free=A, count=A, blocks=64,
            src=A, dst=A, n=A, granted=None, shared=None, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, NULL) for k in ("table", "held", "lens", "parents", "shares", "free", "count", "src", "dst", "n")],
    (dict(batch=0), ARG), (dict(max_blocks=0), ARG), (dict(width=0), ARG), (dict(bt=0), ARG), (dict(blocks=0), ARG),
    (dict(width=3), SHAPE), (dict(width=65), UNSUPPORTED), (dict(batch=4100), UNSUPPORTED),
    (dict(max_blocks=1 << 29), UNSUPPORTED), (dict(blocks=2**31 - 1), UNSUPPORTED), (dict(table=A + 4), ALIGN),
    (dict(shares=A + 4), ALIGN), (dict(granted=A + 4), ALIGN), (dict(shared=A + 4), ALIGN), (dict(dst=A + 4), ALIGN),
    (dict(ws=None), WORKSPACE), (dict(ws=A + 16), ALIGN), (dict(ws_bytes=255), WORKSPACE)])
def test_fork_refusals(change, code):
    assert _call("kv_blocks_fork", FORK, change) == code


def _buffers(*pairs):
    return (beam.block_buffer * len(pairs))(*[beam.block_buffer(*p) for p in pairs])


COPY = dict(bufs=_buffers((A, 64), (2 * A, 4096)), n=2, blocks=10, src=A, dst=A, pairs=5, count=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(bufs=None), NULL), (dict(src=None), NULL), (dict(dst=None), NULL), (dict(bufs=_buffers((A, 64), (None, 64))), NULL),
    (dict(n=0), ARG), (dict(blocks=0), ARG), (dict(pairs=0), ARG), (dict(bufs=_buffers((A, 64), (A, 0))), ARG),
    (dict(bufs=_buffers((A, 64), (A, 24))), ARG), (dict(n=161), UNSUPPORTED),
    (dict(bufs=_buffers((A, 64), (A, 1 << 60)), blocks=100), UNSUPPORTED),
    (dict(bufs=_buffers((A, 1 << 43), (A, 1 << 43)), blocks=1), UNSUPPORTED),
    (dict(bufs=_buffers((A, 64), (A + 16, 64))), ALIGN), (dict(src=A + 4), ALIGN), (dict(dst=A + 4), ALIGN),
    (dict(count=A + 4), ALIGN)])
def test_copy_refusals(change, code):
    assert _call("kv_blocks_copy", COPY, change) == code


COMPACT = dict(table=A, batch=8, max_blocks=10, held=A, keep=32, shares=A, free=A, count=A, blocks=64, moved=A, src=A, dst=A,
               most=32, n=A, done=A, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    *[({k: None}, NULL) for k in ("table", "held", "shares", "free", "count", "moved", "src", "dst", "n", "done")],
    (dict(batch=0), ARG), (dict(max_blocks=0), ARG), (dict(blocks=0), ARG), (dict(keep=-1), ARG), (dict(keep=65), ARG),
    (dict(most=0), ARG), (dict(batch=4097), UNSUPPORTED), (dict(max_blocks=1 << 29), UNSUPPORTED),
    (dict(blocks=2**31 - 1), UNSUPPORTED), (dict(moved=A + 4), ALIGN), (dict(done=A + 4), ALIGN), (dict(ws=None), WORKSPACE),
    (dict(ws=A + 8), ALIGN), (dict(ws_bytes=300), WORKSPACE)])
def test_compact_refusals(change, code):
    assert _call("kv_blocks_compact", COMPACT, change) == code


@pytest.mark.parametrize("args", [(0, 5), (4097, 5), (1, 0), (1, 2**31 - 1)])
def test_workspace_query_refuses(args):
    assert beam.kv_blocks_workspace_bytes(*args) == 0


def test_binding_refuses_tensors_off_the_gpu():
    import torch
    x = torch.zeros((4, 10))
    i = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError):
        beam.beam_select(x, x[:1, :4], x[:1, :4], i, i)
    with pytest.raises(ValueError):
        beam.kv_blocks_compact(i, i, 0, i, i, i, i, i, i, i, i, i)
    with pytest.raises(ValueError):
        beam.BlockBuffers(3, [x])
    with pytest.raises(ValueError):
        beam.BlockBuffers(0, [x])
    with pytest.raises(ValueError):
        beam.BlockBuffers(4, [])


def test_oracle_select_ties_bans_and_ended_beams():
    x = np.zeros((3, 4), np.float32)
    x[1, 2] = -np.inf
    s, p, t = obeam.select(x, np.zeros((1, 3), np.float32), 6, np.array([[False, False, True]]), 1)
    # the ended beam keeps its score 0, then -log 3 of beam 1 (three tokens left), then -log 4 of beam 0
    assert p[0].tolist() == [2, 1, 1, 1, 0, 0] and t[0].tolist() == [1, 0, 1, 3, 0, 1]
    assert np.allclose(s[0], [0, *[-np.log(3)] * 3, *[-np.log(4)] * 2])
    s, p, t = obeam.select(np.full((2, 3), -np.inf), np.zeros((1, 2)), 3)
    assert (s == -np.inf).all() and p[0].tolist() == [0, 0, 0] and t[0].tolist() == [0, 1, 2]


def test_oracle_fork_shares_copies_and_frees():
    # one request of three sequences; the second takes the first's place, the third ends
    table = np.array([[5, 6, -1], [7, 3, -1], [4, -1, -1]])
    r = obeam.fork(table, [2, 2, 1], [20, 32, 9], [0, 0, -1], 3, 16, [0] * 8, [0, 1, 2])
    # 7, 4 and 3 are free: pushed in descending order, the lowest on top; the copy of the last block takes it
    assert r["free"] == [0, 1, 2, 7, 4] and r["pairs"] == [(6, 3)]
    assert r["table"].tolist() == [[5, 6, -1], [5, 3, -1], [-1, -1, -1]]
    assert r["held"] == [2, 2, 0] and r["lens"] == [20, 20, 0] and r["shared"] == [1] and r["granted"] == [1, 1, 1]
    assert r["shares"][5] == 1 and sum(r["shares"]) == 1


def test_oracle_fork_without_free_blocks_goes_on_sharing():
    r = obeam.fork(np.array([[0], [-1]]), [1, 0], [9, 0], [0, 0], 2, 16, [0], [])
    assert r["granted"] == [1, 0] and r["table"].tolist() == [[0], [0]] and r["shares"] == [1] and r["shared"] == [0]


def test_oracle_compact_moves_the_upper_blocks_down():
    r = obeam.compact(np.array([[6, 1], [4, 6]]), [2, 2], 4, [0, 0, 0, 0, 0, 0, 1, 0], [7, 3, 0, 5, 2], 9)
    assert r["pairs"] == [(4, 0), (6, 2)] and r["table"].tolist() == [[2, 1], [0, 2]]
    assert r["free"] == [3] and r["shares"][2] == 1 and r["shares"][6] == 0 and r["done"] == 1
    assert obeam.compact(np.array([[6, 1], [4, 6]]), [2, 2], 4, [0] * 8, [7, 3, 0, 5, 2], 1)["done"] == 0


def _pool(role, fmt=0, per_head=0, blocks=8, heads=2, dim=128):
    return kvq.fp8_pool_init(role, fmt, per_head, blocks, heads, dim, A, 2 * A)


def _group_args():
    return dict(q=A, qs=1024, k=_pool(0), v=_pool(1), table=A, lens=A, shared=A, batch=8, width=4, hq=8, max_blocks=8, most=128,
                out=A, wide=0, scale=0.0, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(v=_pool(0)), ARG), (dict(v=_pool(1, fmt=1)), ARG), (dict(v=_pool(1, heads=4)), SHAPE), (dict(q=None), NULL),
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(shared=None), NULL), (dict(out=None), NULL), (dict(batch=0), ARG),
    (dict(width=0), ARG), (dict(most=0), ARG), (dict(width=3), SHAPE), (dict(hq=7), SHAPE), (dict(batch=4100), UNSUPPORTED),
    (dict(width=65, batch=65), UNSUPPORTED), (dict(hq=130, qs=130 * 128), UNSUPPORTED), (dict(qs=1016), ARG),
    (dict(qs=1028), ARG), (dict(most=129), CAPACITY), (dict(q=A + 8), ALIGN), (dict(shared=A + 4), ALIGN),
    (dict(out=A + 16), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=A + 16), ALIGN), (dict(ws_bytes=1 << 20), WORKSPACE),
    (dict(k=_pool(0, heads=65535), v=_pool(1, heads=65535), batch=4096, hq=65535 * 64, qs=65535 * 64 * 128), UNSUPPORTED),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG)])
def test_group_refusals(change, code):
    assert _call("fp8_group_attention", _group_args(), change) == code


@pytest.mark.parametrize("args", [(0, 1, 2, 8, 128), (8, 3, 2, 8, 128), (8, 0, 2, 8, 128), (65, 65, 2, 8, 128), (8, 4, 0, 8, 128),
                                  (8, 4, 2, 7, 128), (8, 4, 2, 8, 96), (4097, 1, 2, 8, 128), (8, 4, 1, 65, 128),
                                  (4096, 4, 65535, 65535 * 64, 128)])
def test_group_workspace_query_refuses(args):
    assert beam.fp8_group_workspace_bytes(*args) == 0
