"""The speculative-decoding calls without a GPU: exported symbols, refusals (no
kernel is launched), the binding's argument checks, and the oracle's tables."""
import ctypes
import os
import re

import numpy as np
import pytest

from oracle import spec as ospec

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "kvq_spec.h")

kvq = pytest.importorskip("quantized_kv_cache_quant_gb300.kvq", reason="libkvq.so not built")
spec = pytest.importorskip("quantized_kv_cache_quant_gb300.spec")

A = 1 << 20  # a fake, 256-byte aligned address: the checks never read through it
OK, NULL, ARG, SHAPE, CAPACITY, WORKSPACE, UNSUPPORTED, ALIGN = 0, 1, 2, 3, 4, 5, 6, 9


def test_declared_symbols_are_exported_and_bound():
    names = re.findall(r"KVQ_API\s+[\w\s\*]+?\b(\w+)\s*\(", open(HEADER, encoding="utf-8").read())
    assert sorted(names) == sorted(spec.EXPORTED) == sorted(spec._SIG)
    lib = ctypes.CDLL(kvq.LIB_PATH)
    for n in names:
        assert hasattr(lib, n), n


def test_limits_match_the_header():
    text = open(HEADER, encoding="utf-8").read()
    for name, value in (("KVQ_SPEC_MAX_BATCH", spec.MAX_BATCH), ("KVQ_TREE_MAX", spec.TREE_MAX),
                        ("KVQ_TREE_MAX_GQA", spec.TREE_MAX_GQA)):
        assert int(re.search(rf"#define {name}\s+(\d+)", text).group(1)) == value


def _pool(role, fmt=0, per_head=0, blocks=8, heads=2, dim=128):
    return kvq.fp8_pool_init(role, fmt, per_head, blocks, heads, dim, A, 2 * A)


def _call(name, args, change):
    args = dict(args, **change)
    return getattr(kvq._lib, name)(*args.values())


RESIZE = dict(table=A, batch=2, max_blocks=8, held=A, target=A, bt=16, free=A, count=A, blocks=32, granted=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(table=None), NULL), (dict(held=None), NULL), (dict(target=None), NULL), (dict(free=None), NULL),
    (dict(count=None), NULL), (dict(batch=0), ARG), (dict(max_blocks=0), ARG), (dict(bt=0), ARG), (dict(blocks=-1), ARG),
    (dict(batch=4097), UNSUPPORTED), (dict(batch=4096, max_blocks=1 << 20), UNSUPPORTED), (dict(held=A + 4), ALIGN),
    (dict(granted=A + 8), ALIGN)])
def test_resize_refusals(change, code):
    assert _call("kv_blocks_resize", RESIZE, change) == code


MAP = dict(table=A, batch=2, max_blocks=8, seq=A, new=A, bt=16, blocks=32, rows=5, offsets=A, slots=A, ids=None, pos=None,
           stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(table=None), NULL), (dict(seq=None), NULL), (dict(new=None), NULL), (dict(offsets=None), NULL),
    (dict(slots=None), NULL), (dict(rows=0), ARG), (dict(batch=-1), ARG), (dict(bt=0), ARG), (dict(blocks=0), ARG),
    (dict(batch=4097), UNSUPPORTED), (dict(slots=A + 8), ALIGN), (dict(ids=A + 4), ALIGN), (dict(pos=A + 4), ALIGN)])
def test_slot_map_refusals(change, code):
    assert _call("kv_slot_map", MAP, change) == code


def _append_args():
    return dict(k=_pool(0), v=_pool(1), kn=A, ks=256, vn=A, vs=256, slots=A, n=4, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(k=_pool(1)), ARG), (dict(v=_pool(0)), ARG), (dict(v=_pool(1, fmt=1)), ARG), (dict(v=_pool(1, per_head=1)), ARG),
    (dict(v=_pool(1, blocks=9)), SHAPE), (dict(v=_pool(1, heads=1)), SHAPE), (dict(v=_pool(1, dim=64)), SHAPE),
    (dict(k=None), NULL), (dict(kn=None), NULL), (dict(vn=None), NULL), (dict(slots=None), NULL), (dict(n=0), ARG),
    (dict(ks=255), ARG), (dict(ks=248), ARG), (dict(vs=260), ARG), (dict(kn=A + 8), ALIGN), (dict(vn=A + 2), ALIGN),
    (dict(slots=A + 8), ALIGN)])
def test_append_refusals(change, code):
    assert _call("fp8_kv_append", _append_args(), change) == code


def _accept_args():
    return dict(k=_pool(0), v=_pool(1), table=A, batch=2, max_blocks=8, seq=A, path=A, path_len=4, n=A, new=A, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(v=_pool(0)), ARG), (dict(v=_pool(1, blocks=9)), SHAPE), (dict(table=None), NULL), (dict(path=None), NULL),
    (dict(n=None), NULL), (dict(new=None), NULL), (dict(seq=None), NULL), (dict(batch=0), ARG), (dict(path_len=0), ARG),
    (dict(path_len=257), UNSUPPORTED), (dict(batch=4097), UNSUPPORTED), (dict(path=A + 4), ALIGN), (dict(new=A + 4), ALIGN)])
def test_accept_refusals(change, code):
    assert _call("fp8_kv_accept", _accept_args(), change) == code


def _tree_args():
    return dict(q=A, qs=1024, n=10, k=_pool(0), v=_pool(1), table=A, seq=A, offsets=A, mask=A, words=1, batch=2, hq=8,
                max_blocks=8, max_tree=5, max_seq=128, out=A, wide=0, scale=0.0, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(v=_pool(0)), ARG), (dict(v=_pool(1, fmt=1)), ARG), (dict(v=_pool(1, heads=4)), SHAPE), (dict(q=None), NULL),
    (dict(table=None), NULL), (dict(seq=None), NULL), (dict(offsets=None), NULL), (dict(mask=None), NULL),
    (dict(out=None), NULL), (dict(n=0), ARG), (dict(batch=0), ARG), (dict(max_tree=0), ARG), (dict(max_seq=0), ARG),
    (dict(max_tree=257, words=5), UNSUPPORTED), (dict(batch=4097), UNSUPPORTED), (dict(hq=7), SHAPE),
    (dict(hq=130, qs=130 * 128), UNSUPPORTED), (dict(max_tree=65), ARG), (dict(words=0), ARG), (dict(qs=1016), ARG),
    (dict(qs=1028), ARG), (dict(max_seq=129), CAPACITY), (dict(q=A + 8), ALIGN), (dict(mask=A + 8), ALIGN),
    (dict(out=A + 16), ALIGN), (dict(ws=None), WORKSPACE), (dict(ws=A + 16), ALIGN), (dict(ws_bytes=0), WORKSPACE),
    (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG)])
def test_tree_refusals(change, code):
    assert _call("fp8_tree_attention", _tree_args(), change) == code


@pytest.mark.parametrize("args", [(0, 2, 8, 128, 5), (2, 0, 8, 128, 5), (2, 2, 7, 128, 5), (2, 2, 8, 96, 5), (2, 2, 8, 128, 0),
                                  (2, 2, 8, 128, 257), (4097, 2, 8, 128, 5), (2, 1, 65, 128, 5)])
def test_workspace_query_refuses(args):
    assert spec.fp8_tree_workspace_bytes(*args) == 0


def test_binding_refuses_tensors_off_the_gpu():
    import torch
    t = torch.zeros((2, 4), dtype=torch.int32)
    one = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        spec.kv_blocks_resize(t, one, one, 16, one, one[:1])


def test_oracle_resize_restores_the_stack_and_refuses_in_order():
    rng = np.random.default_rng(0)
    free = rng.permutation(40).tolist()
    table, held = np.full((3, 8), -1), np.zeros(3, int)
    t1, h1, f1, g = ospec.resize(table, held, [33, 1, 64], 16, free)
    assert h1.tolist() == [3, 1, 4] and g.tolist() == [1, 1, 1]
    assert t1[0, :3].tolist() == free[::-1][:3] and t1[1, 0] == free[::-1][3]
    t2, h2, f2, _ = ospec.resize(t1, h1, [0, 0, 0], 16, f1)
    assert f2 == free and (t2 == -1).all()
    # 5 free blocks: the second request does not fit, and no later one that grows is served before it
    _, h3, f3, g3 = ospec.resize(table, held, [48, 48, 16], 16, free[:5])
    assert g3.tolist() == [1, 0, 0] and h3.tolist() == [3, 0, 0] and len(f3) == 2


def test_oracle_tree_of_one_node_is_decode():
    from oracle import attention, fp8
    rng = np.random.default_rng(1)
    kv = rng.standard_normal((2, 1, 1, 32, 64)).astype(np.float16)
    table = np.array([[1, 0]])
    pools = [fp8.scatter_paged(fp8.quantize(x, np.float32(0.01)), table, 2, 16) for x in kv]
    q = rng.standard_normal((1, 2, 64)).astype(np.float16)
    got = ospec.tree_attention(q, pools[0], pools[1], np.float32(0.01), np.float32(0.01), "e4m3", table, [20], [0, 1],
                               np.ones((1, 1), bool), 0.125)[0]
    hat = [lambda b, h, p=p: fp8.e4m3_decode(fp8.gather_paged(p, table, b, h, 21)) * np.float64(np.float32(0.01)) for p in pools]
    want = attention.decode_attention(q, hat[0], hat[1], 1, 0.125)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_oracle_tree_row_without_tokens_is_zero_and_nan_stays_masked():
    pool = np.full((1, 1, 16, 64), 0x30, np.uint8)
    pool[0, 0, 1] = 0x7F
    sees = np.array([[0, 0], [1, 0]], bool)
    out = ospec.tree_attention(np.ones((2, 1, 64), np.float16), pool, pool, 1.0, 1.0, "e4m3", np.array([[0]]), [0], [0, 2],
                               sees, 1.0)[0]
    assert (out[0] == 0).all() and np.isfinite(out).all()


def test_oracle_slot_map_cuts_and_pads():
    table = np.array([[3, 1], [0, 9]])
    off, slots, seq, pos = ospec.slot_map(table, [14, 15], [3, 2], 16, 4, 7)
    assert off.tolist() == [0, 3, 5]
    assert slots.tolist() == [62, 63, 16, 15, -1, -1, -1]
    assert seq.tolist() == [0, 0, 0, 1, 1, -1, -1] and pos.tolist() == [14, 15, 16, 15, 16, -1, -1]
    assert ospec.slot_map(table, [0, 0], [3, 3], 16, 4, 4)[0].tolist() == [0, 3, 4]
