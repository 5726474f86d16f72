"""Tree attention with key scales of every sign on the GPU."""
import numpy as np
import pytest

import test_gpu_spec as base
from oracle import spec as ospec
from test_gpu_spec import long_tables  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("gq,nodes", [(2, 5), (4, 30)])
@pytest.mark.parametrize("scales", [(0.01, -0.02, 0.0, -0.0, 1e-39), (-0.005, 0.015, 2e-38, -1e-39, 0.0)])
def test_tree_key_scales_of_every_sign(long_tables, scales, gq, nodes, wide):  # noqa: F811
    """A scale below 0 turns the order of the scores, one of 0 (or one that leaves them below the smallest number) makes
    every seen token weigh the same."""
    import torch
    kvq, spec = base._mods()
    rng = np.random.default_rng(50 + nodes)
    p = base.Pools(rng, 30, 5, 64, "e4m3", True)
    p.scale[0] = np.array(scales, np.float32)
    p.pool[0].scale.copy_(torch.from_numpy(p.scale[0]))
    p.upload()
    seq, trees = [150, 3], [nodes, nodes]
    table = rng.permutation(30)[:24].reshape(2, 12).astype(np.int32)
    sees = base.random_sees(rng, trees)
    q = rng.standard_normal((2 * nodes, 5 * gq, 64)).astype(np.float16)
    got, off = base.run_tree(spec, p, table, seq, trees, sees, q, wide)
    ref, mag, spread, dots = ospec.tree_attention(q, p.nat[0], p.nat[1], p.scale[0], p.scale[1], "e4m3", table, seq, off, sees,
                                                  np.float32(0.125))
    assert np.all(np.abs(got - ref) <= base.tree_bound(mag, spread, dots, ref, wide, 64))
