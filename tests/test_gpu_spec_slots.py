"""Slot maps of lengths outside a table on the GPU: each row's answer goes by its position alone."""
import numpy as np
import pytest

from oracle import spec as ospec
from kvq_helpers import dev, host
from test_gpu_spec import i32

pytestmark = pytest.mark.gpu


def check(table, seq, new, bt, num_blocks, rows):
    import torch
    from quantized_kv_cache_quant_gb300 import spec
    off = torch.empty(len(seq) + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    ids, pos = (torch.empty(rows, dtype=torch.int32, device="cuda") for _ in range(2))
    spec.kv_slot_map(dev(table), i32(seq), i32(new), bt, num_blocks, off, slots, ids, pos)
    for got, want in zip((off, slots, ids, pos), ospec.slot_map(table, seq, new, bt, num_blocks, rows)):
        assert np.array_equal(host(got), want)


@pytest.mark.parametrize("bt", [1, 2, 16])
@pytest.mark.parametrize("shift", range(4))
def test_negative_lengths_do_not_hide_the_positions_behind_them(bt, shift):
    """Position 0 at every place of a thread's four rows, behind 1 to 9 positions below it."""
    table = np.arange(2 * 11, dtype=np.int32).reshape(2, 11)
    for length in range(-9, 0):
        check(table, [0, length], [shift, 20], bt, 22, shift + 20)


def test_positions_beyond_31_bits():
    """Blocks of 2^28 tokens: the table holds more positions than 31 bits name."""
    table = np.arange(2 * 12, dtype=np.int32).reshape(2, 12)
    for length in range(2 ** 31 - 9, 2 ** 31):
        check(table, [2 ** 31 - 3, length], [7, 17], 2 ** 28, 24, 30)
