"""Group attention at the sizes its checks let through: the most sequences, the widest groups, the most heads."""
import numpy as np
import pytest

from test_gpu_group import check_group

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("gq", [64, 33])
def test_widest_groups_with_the_most_heads(gq, wide):
    """64 sequences x 64 heads a kv head: 32 tiles of 128 rows, each of which reads the shared blocks."""
    check_group(np.random.default_rng(gq), 64, [9, 0], [None if n % 9 == 4 else n % 23 for n in range(128)], 1, gq, 64, wide=wide)


@pytest.mark.parametrize("width,gq", [(1, 1), (4, 2), (64, 1), (8, 5)])
def test_the_most_sequences(width, gq):
    rng = np.random.default_rng(width)
    own = [None if rng.random() < 0.2 else int(rng.integers(0, 20)) for _ in range(4096)]
    check_group(rng, width, rng.integers(0, 3, 4096 // width).tolist(), own, 1, gq, 64)


@pytest.mark.parametrize("gq", [1, 17])
def test_many_heads(gq):
    check_group(np.random.default_rng(gq), 2, [3], [17, 2], 96, gq, 64, per_head=True)
