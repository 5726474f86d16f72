"""The oracle's slot map of lengths outside a table."""
import numpy as np

from oracle import spec as ospec


def test_oracle_slot_map_of_a_negative_length_and_of_one_at_31_bits():
    table = np.array([[3, 1], [0, 2]])
    off, slots, seq, pos = ospec.slot_map(table, [-2, 2**31 - 1], [4, 2], 16, 4, 6)
    assert off.tolist() == [0, 4, 6] and seq.tolist() == [0] * 4 + [1] * 2
    assert slots.tolist() == [-1, -1, 48, 49, -1, -1]
    assert pos.tolist() == [-2, -1, 0, 1, 2**31 - 1, -1]
    wide = ospec.slot_map(np.arange(12)[None], [2**31 - 1], [2], 2**28, 12, 2)
    assert wide[1].tolist() == [2**31 - 1, -1] and wide[3].tolist() == [2**31 - 1, -1]
