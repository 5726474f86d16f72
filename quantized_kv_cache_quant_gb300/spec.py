"""Speculative decoding over the paged FP8 cache (the C calls of include/kvq_spec.h).

One serving step that verifies drafted tokens: ``kv_blocks_resize`` (the block
tables grow), ``kv_slot_map`` (each new token's place), ``fp8_kv_append`` (keys
and values into the pools), ``fp8_tree_attention`` (the drafted tokens attend
over the cache and, through the tree's mask, to one another), ``fp8_kv_accept``
(the accepted path moves to the end of the sequence), ``kv_blocks_resize`` (what
only rejected tokens held comes back). Functions of the C names take torch
tensors and check their types, layouts and device; shapes come from the tensors.
All work runs in the library's kernels on ``stream`` (default: the current
stream); nothing waits or copies to the host, so a step captures into a graph.
"""
from __future__ import annotations

import ctypes

import torch

from . import kvq
from .kvq import _check, _lib, _P_F8, _stream, c_f32, c_i32, c_sz, c_vp

c_i64 = ctypes.c_int64

MAX_BATCH = 4096      # requests of one call
TREE_MAX = 256        # nodes of one request's tree
TREE_MAX_GQA = 64     # query heads per kv head in tree attention

EXPORTED = ("kv_blocks_resize", "kv_slot_map", "fp8_kv_append", "fp8_kv_accept", "fp8_tree_workspace_bytes",
            "fp8_tree_attention")

_SIG = {
    "kv_blocks_resize": ([c_vp, c_i32, c_i32, c_vp, c_vp, c_i32, c_vp, c_vp, c_i32, c_vp, c_vp], ctypes.c_int),
    "kv_slot_map": ([c_vp, c_i32, c_i32, c_vp, c_vp, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp, c_vp], ctypes.c_int),
    "fp8_kv_append": ([_P_F8, _P_F8, c_vp, c_i64, c_vp, c_i64, c_vp, c_i32, c_vp], ctypes.c_int),
    "fp8_kv_accept": ([_P_F8, _P_F8, c_vp, c_i32, c_i32, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp], ctypes.c_int),
    "fp8_tree_workspace_bytes": ([c_i32, c_i32, c_i32, c_i32, c_i32], c_sz),
    "fp8_tree_attention": ([c_vp, c_i64, c_i32, _P_F8, _P_F8, c_vp, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_i32,
                            c_i32, c_vp, c_i32, c_f32, c_vp, c_sz, c_vp], ctypes.c_int),
}
for _name, (_args, _res) in _SIG.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


# A call's checks cost more host time than the launch itself when each one builds shapes and devices, so they
# compare plain numbers and leave the wording of a refusal to _refuse.
_I32, _I64, _F16 = torch.int32, torch.int64, torch.float16
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _refuse(name: str, t, dtype, n, dev) -> None:
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} expected, not {t.dtype}")
    if t.numel() != n:
        raise ValueError(f"{name}: {n} elements expected, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor expected")
    raise ValueError(f"{name}: on {t.device}, not on cuda:{dev}")


def _arg(name: str, t, dtype, n: int, dev: int) -> int:
    """The address of a contiguous tensor of n elements of this type on device dev."""
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        _refuse(name, t, dtype, n, dev)
    return t.data_ptr()


def _rows(name: str, t, n, heads: int, dim: int, dev: int):
    """(address, row stride) of fp16 rows [n, heads, dim] whose rows are contiguous and may lie apart."""
    if t.dtype is not _F16:
        raise TypeError(f"{name}: {_F16} expected, not {t.dtype}")
    if t.shape != (n, heads, dim):
        raise ValueError(f"{name}: shape {(n, heads, dim)} expected, not {tuple(t.shape)}")
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != dim):
        raise ValueError(f"{name}: contiguous [heads, dim] rows expected")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, not on cuda:{dev}")
    return t.data_ptr(), row if n > 1 else heads * dim


def _here(t) -> int:
    """The tensor's device, which has to be the current one: the kernels launch there."""
    dev = t.get_device()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"tensors have to be on the current CUDA device, not on {t.device}")
    return dev


def _on(stream, dev: int):
    if stream is None and _current_stream is not None:
        return _current_stream(dev)
    return _stream(stream)


def _table(t):
    """(batch, max_blocks) of a block table."""
    if t.dim() != 2:
        raise ValueError(f"block_table: two dimensions expected, not {tuple(t.shape)}")
    return t.shape


def kv_blocks_resize(block_table, n_held, target_tokens, block_tokens: int, free_blocks, free_count, granted=None,
                     stream=None) -> None:
    """Give request b the blocks that ``target_tokens[b]`` tokens need, in place:
    shrinks first, then grows in order of b while free blocks last.
    block_table int32 [B, max_blocks], n_held / target_tokens int32 [B],
    free_blocks int32 [num_blocks] (a stack) with free_count int32 [1], granted
    int32 [B] (written 1 or 0) or None."""
    d = _here(block_table)
    b, width = _table(block_table)
    blocks = free_blocks.numel()
    code = _lib.kv_blocks_resize(
        _arg("block_table", block_table, _I32, b * width, d), b, width, _arg("n_held", n_held, _I32, b, d),
        _arg("target_tokens", target_tokens, _I32, b, d), block_tokens, _arg("free_blocks", free_blocks, _I32, blocks, d),
        _arg("free_count", free_count, _I32, 1, d), blocks,
        None if granted is None else _arg("granted", granted, _I32, b, d), _on(stream, d))
    if code:
        _check(code, "kv_blocks_resize")


def kv_slot_map(block_table, seq_lens, new_lens, block_tokens: int, num_blocks: int, offsets, slots, seq_ids=None,
                positions=None, stream=None) -> None:
    """The slots of each request's new tokens, flattened over requests: writes
    offsets int32 [B + 1], slots int64 [N] and, where given, seq_ids and
    positions int32 [N]; rows behind the last request become -1."""
    d = _here(block_table)
    b, width = _table(block_table)
    n = slots.numel()
    code = _lib.kv_slot_map(
        _arg("block_table", block_table, _I32, b * width, d), b, width, _arg("seq_lens", seq_lens, _I32, b, d),
        _arg("new_lens", new_lens, _I32, b, d), block_tokens, num_blocks, n, _arg("offsets", offsets, _I32, b + 1, d),
        _arg("slots", slots, _I64, n, d), None if seq_ids is None else _arg("seq_ids", seq_ids, _I32, n, d),
        None if positions is None else _arg("positions", positions, _I32, n, d), _on(stream, d))
    if code:
        _check(code, "kv_slot_map")


def fp8_kv_append(k_pool, v_pool, k_new, v_new, slots, stream=None) -> None:
    """Quantize tokens k_new, v_new fp16 [N, H, D] (rows may lie apart) with the
    pools' scales into the rows that slots int64 [N] names (-1: skipped)."""
    d = _here(k_new)
    n, h, dim = slots.numel(), k_pool.kv_heads, k_pool.head_dim
    kp, ks = _rows("k_new", k_new, n, h, dim, d)
    vp, vs = _rows("v_new", v_new, n, h, dim, d)
    code = _lib.fp8_kv_append(k_pool, v_pool, kp, ks, vp, vs, _arg("slots", slots, _I64, n, d), n, _on(stream, d))
    if code:
        _check(code, "fp8_kv_append")


def fp8_kv_accept(k_pool, v_pool, block_table, seq_lens, path, n_accepted, new_lens, stream=None) -> None:
    """Move the accepted nodes' rows (path int32 [B, P], ascending; the first
    n_accepted[b] of a row count) to the end of each sequence and write
    new_lens = seq_lens + n_accepted (new_lens may be seq_lens)."""
    d = _here(block_table)
    b, width = _table(block_table)
    if path.dim() != 2 or path.shape[0] != b:
        raise ValueError(f"path: shape ({b}, P) expected, not {tuple(path.shape)}")
    p = path.shape[1]
    code = _lib.fp8_kv_accept(
        k_pool, v_pool, _arg("block_table", block_table, _I32, b * width, d), b, width,
        _arg("seq_lens", seq_lens, _I32, b, d), _arg("path", path, _I32, b * p, d), p,
        _arg("n_accepted", n_accepted, _I32, b, d), _arg("new_lens", new_lens, _I32, b, d), _on(stream, d))
    if code:
        _check(code, "fp8_kv_accept")


def fp8_tree_workspace_bytes(batch: int, kv_heads: int, q_heads: int, head_dim: int, max_tree: int) -> int:
    return int(_lib.fp8_tree_workspace_bytes(batch, kv_heads, q_heads, head_dim, max_tree))


def fp8_tree_attention(q, k_pool, v_pool, block_table, seq_lens, tree_offsets, tree_mask, max_tree: int,
                       max_seq_len: int, out, softmax_scale: float, ws, stream=None) -> None:
    """Attention of each request's tree over its cached tokens and, through
    tree_mask int64 [N, words] (bit j: node j of the same request is seen), its
    own nodes, whose keys and values fp8_kv_append has written at positions
    seq_lens[b] + j. q fp16 [N, Hq, D] (rows may lie apart); out fp16 or fp32
    [N, Hq, D]; tree_offsets int32 [B + 1]; ws uint8, zeroed once, at least
    fp8_tree_workspace_bytes."""
    d = _here(q)
    n, hq, dim = q.shape
    qp, qs = _rows("q", q, n, hq, k_pool.head_dim, d)
    b, width = _table(block_table)
    if tree_mask.dim() != 2 or tree_mask.shape[0] != n:
        raise ValueError(f"tree_mask: shape ({n}, words) expected, not {tuple(tree_mask.shape)}")
    if out.shape != q.shape:
        raise ValueError(f"out: shape {tuple(q.shape)} expected, not {tuple(out.shape)}")
    words, wide, size = tree_mask.shape[1], out.dtype is torch.float32, ws.numel()
    code = _lib.fp8_tree_attention(
        qp, qs, n, k_pool, v_pool, _arg("block_table", block_table, _I32, b * width, d),
        _arg("seq_lens", seq_lens, _I32, b, d), _arg("tree_offsets", tree_offsets, _I32, b + 1, d),
        _arg("tree_mask", tree_mask, _I64, n * words, d), words, b, hq, width, max_tree, max_seq_len,
        _arg("out", out, torch.float32 if wide else _F16, n * hq * dim, d), int(wide), softmax_scale,
        _arg("ws", ws, torch.uint8, size, d), size, _on(stream, d))
    if code:
        _check(code, "fp8_tree_attention")


class BlockTables:
    """Block tables of a batch with the stack of free blocks, in device memory owned by PyTorch."""

    def __init__(self, batch: int, max_blocks: int, num_blocks: int, block_tokens: int = 16, device="cuda"):
        self.block_tokens, self.num_blocks = block_tokens, num_blocks
        i32 = dict(dtype=torch.int32, device=device)
        self.table = torch.full((batch, max_blocks), -1, **i32)
        self.n_held = torch.zeros(batch, **i32)
        # block 0 on top of the stack
        self.free_blocks = torch.arange(num_blocks - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), num_blocks, **i32)
        self.granted = torch.zeros(batch, **i32)

    def resize(self, target_tokens, stream=None):
        """Hold what target_tokens int32 [B] tokens need; returns `granted` (the instance's own buffer)."""
        kv_blocks_resize(self.table, self.n_held, target_tokens, self.block_tokens, self.free_blocks, self.free_count,
                         self.granted, stream)
        return self.granted

    def slot_map(self, seq_lens, new_lens, offsets, slots, seq_ids=None, positions=None, stream=None):
        kv_slot_map(self.table, seq_lens, new_lens, self.block_tokens, self.num_blocks, offsets, slots, seq_ids,
                    positions, stream)


def tree_workspace(batch: int, kv_heads: int, q_heads: int, head_dim: int, max_tree: int, device="cuda"):
    """A zeroed workspace of fp8_tree_attention for these shapes."""
    n = fp8_tree_workspace_bytes(batch, kv_heads, q_heads, head_dim, max_tree)
    if n == 0:
        raise kvq.KvqError(6, "fp8_tree_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def pack_tree_mask(sees):
    """Mask words int64 [N, words] from a boolean [N, nodes] (column j: node j of the row's own request)."""
    n, nodes = sees.shape
    words = -(-nodes // 64)
    bits = torch.zeros((n, words * 64), dtype=torch.int64, device=sees.device)
    bits[:, :nodes] = sees
    # 63 shifted left wraps to the sign bit, as the word's top bit should
    return (bits.view(n, words, 64) << torch.arange(64, device=sees.device)).sum(-1)
