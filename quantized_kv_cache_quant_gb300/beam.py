"""Beam search and parallel sampling over the paged caches (the C calls of include/kvq_beam.h).

One step that keeps several continuations of each request: ``beam_select`` (the
best candidates from the logits), ``kv_blocks_fork`` (the block tables follow
the parents; full blocks are shared), ``kv_blocks_copy`` (partly filled last
blocks, in every layer's pools), then ``kv_blocks_resize_shared``,
``spec.kv_slot_map`` and ``spec.fp8_kv_append`` for the new tokens and
``fp8_group_attention`` (decode attention that reads the blocks a request's
sequences share once). ``kv_blocks_compact`` empties the end of a pool.
Functions of the C names take torch tensors and check their types, layouts and
device; shapes come from the tensors. All work runs in the library's kernels on
``stream`` (default: the current stream); nothing waits or copies to the host,
so a step captures into a graph.
"""
from __future__ import annotations

import ctypes

import torch

from . import kvq
from .kvq import _check, _lib, _P_F8, c_f32, c_i32, c_sz, c_vp
from .spec import _F16, _I32, _arg, _here, _on, _rows, _table, BlockTables, c_i64

MAX_WIDTH = 64        # sequences of a request
MAX_OUT = 128         # candidates of a request
COPY_MAX_BUFFERS = 160
LOGITS = {torch.float16: 0, torch.float32: 1, torch.bfloat16: 2}

EXPORTED = ("beam_select", "kv_blocks_workspace_bytes", "kv_blocks_fork", "kv_blocks_resize_shared", "kv_blocks_copy",
            "kv_blocks_compact", "fp8_group_workspace_bytes", "fp8_group_attention")


class block_buffer(ctypes.Structure):
    _fields_ = [("base", c_vp), ("block_bytes", c_i64)]


_SIG = {
    "beam_select": ([c_vp, c_i32, c_i64, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_vp, c_vp, c_vp], ctypes.c_int),
    "kv_blocks_workspace_bytes": ([c_i32, c_i32], c_sz),
    "kv_blocks_fork": ([c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_i32, c_i32, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_vp,
                        c_vp, c_vp, c_sz, c_vp], ctypes.c_int),
    "kv_blocks_resize_shared": ([c_vp, c_i32, c_i32, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp], ctypes.c_int),
    "kv_blocks_copy": ([ctypes.POINTER(block_buffer), c_i32, c_i32, c_vp, c_vp, c_i32, c_vp, c_vp], ctypes.c_int),
    "kv_blocks_compact": ([c_vp, c_i32, c_i32, c_vp, c_i32, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp, c_i32, c_vp, c_vp, c_vp,
                           c_sz, c_vp], ctypes.c_int),
    "fp8_group_workspace_bytes": ([c_i32, c_i32, c_i32, c_i32, c_i32], c_sz),
    "fp8_group_attention": ([c_vp, c_i64, _P_F8, _P_F8, c_vp, c_vp, c_vp, c_i32, c_i32, c_i32, c_i32, c_i32, c_vp, c_i32, c_f32,
                             c_vp, c_sz, c_vp], ctypes.c_int),
}
for _name, (_args, _res) in _SIG.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


def beam_select(logits, scores, out_scores, out_parents, out_tokens, finished=None, end_token: int = -1,
                stream=None) -> None:
    """The best candidates of each request by scores[i] + log_softmax(logits[i])[t].
    logits fp16, fp32 or bf16 [R * W, V] (rows may lie apart), scores fp32 [R, W];
    writes out_scores fp32, out_parents int32 (i) and out_tokens int32 (t), each
    [R, n]: best first, those of one beam in the order of their logits, equal
    logits by the lower t, equal scores of different beams by the lower i.
    finished bool or uint8 [R, W] or None: beams that have ended offer
    (end_token, scores[i])."""
    d = _here(logits)
    if logits.dtype not in LOGITS:
        raise TypeError(f"logits: fp16, fp32 or bf16 expected, not {logits.dtype}")
    if scores.dim() != 2 or out_tokens.dim() != 2 or out_tokens.shape[0] != scores.shape[0]:
        raise ValueError(f"scores [R, W] and out_tokens [R, n] expected, not {tuple(scores.shape)} and {tuple(out_tokens.shape)}")
    (r, w), n = scores.shape, out_tokens.shape[1]
    if logits.dim() != 2 or logits.shape[0] != r * w or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits: [{r * w}, V] with contiguous rows expected, not {tuple(logits.shape)}")
    v = logits.shape[1]
    end = None
    if finished is not None:
        end = _arg("finished", finished, torch.bool if finished.dtype is torch.bool else torch.uint8, r * w, d)
    code = _lib.beam_select(
        logits.data_ptr(), LOGITS[logits.dtype], logits.stride(0) if r * w > 1 else v,
        _arg("scores", scores, torch.float32, r * w, d), end, end_token, r, w, v, n,
        _arg("out_scores", out_scores, torch.float32, r * n, d), _arg("out_parents", out_parents, _I32, r * n, d),
        _arg("out_tokens", out_tokens, _I32, r * n, d), _on(stream, d))
    if code:
        _check(code, "beam_select")


def kv_blocks_workspace_bytes(groups: int, num_blocks: int) -> int:
    return int(_lib.kv_blocks_workspace_bytes(groups, num_blocks))


def blocks_workspace(groups: int, num_blocks: int, device="cuda"):
    """A zeroed workspace of kv_blocks_fork (this many requests) and kv_blocks_compact, for pools of up to num_blocks blocks."""
    n = kv_blocks_workspace_bytes(groups, num_blocks)
    if n == 0:
        raise kvq.KvqError(6, "kv_blocks_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def kv_blocks_fork(block_table, n_held, seq_lens, parents, width: int, block_tokens: int, shares, free_blocks, free_count,
                   copy_src, copy_dst, copy_count, ws, granted=None, shared_blocks=None, stream=None) -> None:
    """Every sequence becomes a copy of its parent, in place (parents int32 [B]:
    a place within the request of ``width`` sequences; any other value empties
    the sequence). block_table int32 [B, max_blocks], n_held / seq_lens int32
    [B], shares and free_blocks int32 [num_blocks], free_count int32 [1] are
    updated; copy_src / copy_dst int32 [B] and copy_count int32 [1] receive the
    blocks to copy; granted int32 [B] and shared_blocks int32 [B / width] may be
    None; ws uint8, zeroed once, at least kv_blocks_workspace_bytes."""
    d = _here(block_table)
    b, max_blocks = _table(block_table)
    blocks, size = free_blocks.numel(), ws.numel()
    code = _lib.kv_blocks_fork(
        _arg("block_table", block_table, _I32, b * max_blocks, d), b, max_blocks, _arg("n_held", n_held, _I32, b, d),
        _arg("seq_lens", seq_lens, _I32, b, d), _arg("parents", parents, _I32, b, d), width, block_tokens,
        _arg("shares", shares, _I32, blocks, d), _arg("free_blocks", free_blocks, _I32, blocks, d),
        _arg("free_count", free_count, _I32, 1, d), blocks, _arg("copy_src", copy_src, _I32, b, d),
        _arg("copy_dst", copy_dst, _I32, b, d), _arg("copy_count", copy_count, _I32, 1, d),
        None if granted is None else _arg("granted", granted, _I32, b, d),
        None if shared_blocks is None else _arg("shared_blocks", shared_blocks, _I32, b // max(width, 1), d),
        _arg("ws", ws, torch.uint8, size, d), size, _on(stream, d))
    if code:
        _check(code, "kv_blocks_fork")


def kv_blocks_resize_shared(block_table, n_held, target_tokens, block_tokens: int, shares, free_blocks, free_count,
                            granted=None, stream=None) -> None:
    """``spec.kv_blocks_resize`` on tables that may share blocks: a sequence that
    would release a block with shares above 0 (int32 [num_blocks]) is refused
    (granted 0) and left as it was. Shortened sequences: lower seq_lens, then
    kv_blocks_fork with every sequence its own parent."""
    d = _here(block_table)
    b, width = _table(block_table)
    blocks = free_blocks.numel()
    code = _lib.kv_blocks_resize_shared(
        _arg("block_table", block_table, _I32, b * width, d), b, width, _arg("n_held", n_held, _I32, b, d),
        _arg("target_tokens", target_tokens, _I32, b, d), block_tokens, _arg("shares", shares, _I32, blocks, d),
        _arg("free_blocks", free_blocks, _I32, blocks, d), _arg("free_count", free_count, _I32, 1, d), blocks,
        None if granted is None else _arg("granted", granted, _I32, b, d), _on(stream, d))
    if code:
        _check(code, "kv_blocks_resize_shared")


class BlockBuffers:
    """The memory of pools with num_blocks blocks each (fp8_pool's and nvfp4_pool's, all layers' keys and values), as
    kv_blocks_copy takes it. Made once; the tensors are kept alive."""

    def __init__(self, num_blocks: int, tensors):
        self.num_blocks, self.tensors = num_blocks, list(tensors)
        if num_blocks <= 0:
            raise ValueError(f"num_blocks: above 0 expected, not {num_blocks}")
        if not 0 < len(self.tensors) <= COPY_MAX_BUFFERS:
            raise ValueError(f"1 to {COPY_MAX_BUFFERS} buffers expected, not {len(self.tensors)}")
        self.array = (block_buffer * len(self.tensors))()
        self.device = self.tensors[0].get_device()
        for at, t in zip(self.array, self.tensors):
            size = t.numel() * t.element_size()
            if not t.is_contiguous() or t.get_device() != self.device or size % num_blocks:
                raise ValueError(f"contiguous buffers of {num_blocks} blocks on one device expected")
            at.base, at.block_bytes = t.data_ptr(), size // num_blocks


def kv_blocks_copy(buffers: BlockBuffers, src, dst, count=None, stream=None) -> None:
    """Copy block src[i] to block dst[i] (int32 [N]; the first count[0] of them
    where count int32 [1] is given) in each of the buffers."""
    d = _here(src)
    if buffers.device != d:
        raise ValueError(f"buffers: on device {buffers.device}, not on cuda:{d}")
    n = src.numel()
    code = _lib.kv_blocks_copy(
        buffers.array, len(buffers.tensors), buffers.num_blocks, _arg("src", src, _I32, n, d),
        _arg("dst", dst, _I32, n, d), n, None if count is None else _arg("count", count, _I32, 1, d), _on(stream, d))
    if code:
        _check(code, "kv_blocks_copy")


def kv_blocks_compact(block_table, n_held, keep_blocks: int, shares, free_blocks, free_count, moved_to, copy_src, copy_dst,
                      copy_count, done, ws, stream=None) -> None:
    """Move the used blocks from keep_blocks on to free ones below: updates
    block_table int32 [B, max_blocks] (n_held int32 [B] entries a row), shares and
    free_blocks int32 [num_blocks] and free_count int32 [1]; writes moved_to int32
    [num_blocks], the pairs to copy (copy_src / copy_dst int32 [N], copy_count int32
    [1]) and done int32 [1] (0: too little room, nothing changed)."""
    d = _here(block_table)
    b, max_blocks = _table(block_table)
    blocks, n, size = free_blocks.numel(), copy_src.numel(), ws.numel()
    code = _lib.kv_blocks_compact(
        _arg("block_table", block_table, _I32, b * max_blocks, d), b, max_blocks, _arg("n_held", n_held, _I32, b, d),
        keep_blocks, _arg("shares", shares, _I32, blocks, d), _arg("free_blocks", free_blocks, _I32, blocks, d),
        _arg("free_count", free_count, _I32, 1, d), blocks, _arg("moved_to", moved_to, _I32, blocks, d),
        _arg("copy_src", copy_src, _I32, n, d), _arg("copy_dst", copy_dst, _I32, n, d), n,
        _arg("copy_count", copy_count, _I32, 1, d), _arg("done", done, _I32, 1, d), _arg("ws", ws, torch.uint8, size, d), size,
        _on(stream, d))
    if code:
        _check(code, "kv_blocks_compact")


def fp8_group_workspace_bytes(batch: int, width: int, kv_heads: int, q_heads: int, head_dim: int) -> int:
    return int(_lib.fp8_group_workspace_bytes(batch, width, kv_heads, q_heads, head_dim))


def group_workspace(batch: int, kv_heads: int, q_heads: int, head_dim: int, width: int, device="cuda"):
    """A zeroed workspace of fp8_group_attention for these shapes."""
    n = fp8_group_workspace_bytes(batch, width, kv_heads, q_heads, head_dim)
    if n == 0:
        raise kvq.KvqError(6, "fp8_group_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def fp8_group_attention(q, k_pool, v_pool, block_table, seq_lens, shared_blocks, width: int, max_seq_len: int, out,
                        softmax_scale: float, ws, stream=None) -> None:
    """Decode attention of sequences in groups of ``width`` whose first
    shared_blocks int32 [B / width] table entries are the same: these blocks are
    read once a group (once for every 128 query rows, width * Hq / H, of a kv
    head). q fp16 [B, Hq, D] (rows may lie apart); out fp16 or fp32 [B, Hq, D]
    (fp32 is the more exact, and slower above 16 such rows); block_table int32
    [B, max_blocks]; seq_lens int32 [B] (0: an empty sequence, whose output is 0);
    ws uint8, zeroed once, at least fp8_group_workspace_bytes."""
    d = _here(q)
    if q.dim() != 3:
        raise ValueError(f"q: [B, Hq, D] expected, not {tuple(q.shape)}")
    n, hq, dim = q.shape
    qp, qs = _rows("q", q, n, hq, k_pool.head_dim, d)
    b, max_blocks = _table(block_table)
    if b != n:
        raise ValueError(f"block_table: {n} rows expected, not {b}")
    if out.shape != q.shape:
        raise ValueError(f"out: shape {tuple(q.shape)} expected, not {tuple(out.shape)}")
    wide, size = out.dtype is torch.float32, ws.numel()
    code = _lib.fp8_group_attention(
        qp, qs, k_pool, v_pool, _arg("block_table", block_table, _I32, b * max_blocks, d),
        _arg("seq_lens", seq_lens, _I32, b, d), _arg("shared_blocks", shared_blocks, _I32, b // max(width, 1), d), b, width, hq,
        max_blocks, max_seq_len, _arg("out", out, torch.float32 if wide else _F16, n * hq * dim, d), int(wide), softmax_scale,
        _arg("ws", ws, torch.uint8, size, d), size, _on(stream, d))
    if code:
        _check(code, "fp8_group_attention")


class BeamTables(BlockTables):
    """Block tables of requests with ``width`` sequences each, which may share blocks: BlockTables with the counts of
    references, the lists of blocks to copy and what fp8_group_attention goes by. ``resize`` refuses a sequence that would
    release a block that others hold: lower ``seq_lens`` and ``fork`` every sequence to itself."""

    def __init__(self, requests: int, width: int, max_blocks: int, num_blocks: int, block_tokens: int = 16, device="cuda"):
        super().__init__(requests * width, max_blocks, num_blocks, block_tokens, device)
        i32 = dict(dtype=torch.int32, device=device)
        self.width = width
        self.seq_lens = torch.zeros(requests * width, **i32)
        self.shares = torch.zeros(num_blocks, **i32)
        self.shared_blocks = torch.zeros(requests, **i32)
        most = max(requests * width, num_blocks // 2)
        self.copy_src, self.copy_dst = torch.zeros(most, **i32), torch.zeros(most, **i32)
        self.copy_count, self.done = torch.zeros(1, **i32), torch.zeros(1, **i32)
        self.moved_to = torch.empty(num_blocks, **i32)
        self.ws = blocks_workspace(requests, num_blocks, device)

    def resize(self, target_tokens, stream=None):
        """Hold what target_tokens int32 [B] tokens need; returns `granted` (the instance's own buffer)."""
        kv_blocks_resize_shared(self.table, self.n_held, target_tokens, self.block_tokens, self.shares, self.free_blocks,
                                self.free_count, self.granted, stream)
        return self.granted

    def fork(self, parents, stream=None):
        """Sequences follow their parents (int32 [requests * width]); copy() has to follow before the next append.
        Returns `granted` (the instance's own buffer)."""
        b = self.table.shape[0]
        kv_blocks_fork(self.table, self.n_held, self.seq_lens, parents, self.width, self.block_tokens, self.shares,
                       self.free_blocks, self.free_count, self.copy_src[:b], self.copy_dst[:b], self.copy_count, self.ws,
                       self.granted, self.shared_blocks, stream)
        return self.granted

    def compact(self, keep_blocks: int, stream=None):
        """Empty the pool's blocks from keep_blocks on; copy() has to follow. Returns `done` (the instance's own buffer)."""
        kv_blocks_compact(self.table, self.n_held, keep_blocks, self.shares, self.free_blocks, self.free_count,
                          self.moved_to, self.copy_src, self.copy_dst, self.copy_count, self.done, self.ws, stream)
        return self.done

    def copy(self, buffers: BlockBuffers, stream=None):
        """Carry out the copies of the last fork or compact."""
        kv_blocks_copy(buffers, self.copy_src, self.copy_dst, self.copy_count, stream)
