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


def _arg(name: str, t, dtype, shape, device) -> int:
    """The address of a contiguous tensor of this type, shape (None: any size) and device."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} expected, not {t.dtype}")
    s = t.shape
    if len(s) != len(shape) or any(w is not None and n != w for n, w in zip(s, shape)):
        raise ValueError(f"{name}: shape {tuple(shape)} expected (None: any), not {tuple(s)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor expected")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")
    return t.data_ptr()


def _rows(name: str, t, heads: int, dim: int, device):
    """(address, row stride) of fp16 rows [N, heads, dim] whose rows are contiguous and may lie apart."""
    if t.dtype is not torch.float16:
        raise TypeError(f"{name}: torch.float16 expected, not {t.dtype}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name}: shape (N, {heads}, {dim}) expected, not {tuple(t.shape)}")
    row, head, one = t.stride()
    if one != 1 or (heads > 1 and head != dim):
        raise ValueError(f"{name}: contiguous [heads, dim] rows expected")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, not on {device}")
    return t.data_ptr(), row if t.shape[0] > 1 else max(row, heads * dim)


def _here(t) -> torch.device:
    """The tensor's device, which has to be the current one: the kernels launch there."""
    d = t.device
    if d.type != "cuda" or d.index != torch.cuda.current_device():
        raise ValueError(f"tensors have to be on the current CUDA device, not on {d}")
    return d


def kv_blocks_resize(block_table, n_held, target_tokens, block_tokens: int, free_blocks, free_count, granted=None,
                     stream=None) -> None:
    """Give request b the blocks that ``target_tokens[b]`` tokens need, in place:
    shrinks first, then grows in order of b while free blocks last.
    block_table int32 [B, max_blocks], n_held / target_tokens int32 [B],
    free_blocks int32 [num_blocks] (a stack) with free_count int32 [1], granted
    int32 [B] (written 1 or 0) or None."""
    d = _here(block_table)
    i32 = torch.int32
    b, width = block_table.shape
    _check(_lib.kv_blocks_resize(
        _arg("block_table", block_table, i32, (b, width), d), b, width, _arg("n_held", n_held, i32, (b,), d),
        _arg("target_tokens", target_tokens, i32, (b,), d), block_tokens,
        _arg("free_blocks", free_blocks, i32, (None,), d), _arg("free_count", free_count, i32, (1,), d),
        free_blocks.shape[0], None if granted is None else _arg("granted", granted, i32, (b,), d), _stream(stream)),
        "kv_blocks_resize")


def kv_slot_map(block_table, seq_lens, new_lens, block_tokens: int, num_blocks: int, offsets, slots, seq_ids=None,
                positions=None, stream=None) -> None:
    """The slots of each request's new tokens, flattened over requests: writes
    offsets int32 [B + 1], slots int64 [N] and, where given, seq_ids and
    positions int32 [N]; rows behind the last request become -1."""
    d = _here(block_table)
    i32 = torch.int32
    b, width = block_table.shape
    n = slots.shape[0]
    _check(_lib.kv_slot_map(
        _arg("block_table", block_table, i32, (b, width), d), b, width, _arg("seq_lens", seq_lens, i32, (b,), d),
        _arg("new_lens", new_lens, i32, (b,), d), block_tokens, num_blocks, n,
        _arg("offsets", offsets, i32, (b + 1,), d), _arg("slots", slots, torch.int64, (n,), d),
        None if seq_ids is None else _arg("seq_ids", seq_ids, i32, (n,), d),
        None if positions is None else _arg("positions", positions, i32, (n,), d), _stream(stream)), "kv_slot_map")


def fp8_kv_append(k_pool, v_pool, k_new, v_new, slots, stream=None) -> None:
    """Quantize tokens k_new, v_new fp16 [N, H, D] (rows may lie apart) with the
    pools' scales into the rows that slots int64 [N] names (-1: skipped)."""
    d = _here(k_new)
    kp, ks = _rows("k_new", k_new, k_pool.kv_heads, k_pool.head_dim, d)
    vp, vs = _rows("v_new", v_new, k_pool.kv_heads, k_pool.head_dim, d)
    n = k_new.shape[0]
    if v_new.shape[0] != n:
        raise ValueError(f"v_new: {n} rows expected, not {v_new.shape[0]}")
    _check(_lib.fp8_kv_append(k_pool, v_pool, kp, ks, vp, vs, _arg("slots", slots, torch.int64, (n,), d), n,
                              _stream(stream)), "fp8_kv_append")


def fp8_kv_accept(k_pool, v_pool, block_table, seq_lens, path, n_accepted, new_lens, stream=None) -> None:
    """Move the accepted nodes' rows (path int32 [B, P], ascending; the first
    n_accepted[b] of a row count) to the end of each sequence and write
    new_lens = seq_lens + n_accepted (new_lens may be seq_lens)."""
    d = _here(block_table)
    i32 = torch.int32
    b, width = block_table.shape
    _check(_lib.fp8_kv_accept(
        k_pool, v_pool, _arg("block_table", block_table, i32, (b, width), d), b, width,
        _arg("seq_lens", seq_lens, i32, (b,), d), _arg("path", path, i32, (b, None), d), path.shape[1],
        _arg("n_accepted", n_accepted, i32, (b,), d), _arg("new_lens", new_lens, i32, (b,), d), _stream(stream)),
        "fp8_kv_accept")


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
    i32 = torch.int32
    n, hq, dim = q.shape
    qp, qs = _rows("q", q, hq, k_pool.head_dim, d)
    b, width = block_table.shape
    wide = out.dtype is torch.float32
    _check(_lib.fp8_tree_attention(
        qp, qs, n, k_pool, v_pool, _arg("block_table", block_table, i32, (b, width), d),
        _arg("seq_lens", seq_lens, i32, (b,), d), _arg("tree_offsets", tree_offsets, i32, (b + 1,), d),
        _arg("tree_mask", tree_mask, torch.int64, (n, None), d), tree_mask.shape[1], b, hq, width, max_tree, max_seq_len,
        _arg("out", out, torch.float32 if wide else torch.float16, (n, hq, dim), d), int(wide), softmax_scale,
        _arg("ws", ws, torch.uint8, (None,), d), ws.shape[0], _stream(stream)), "fp8_tree_attention")


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
