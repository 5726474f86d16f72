"""Tree attention on the GPU where one pair's result meets the next pair's work in a thread block."""
import numpy as np
import pytest

import test_gpu_spec as base
from kvq_helpers import dev
from test_gpu_spec import long_tables  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,wide", [(128, False), (64, True)])
def test_tree_pair_of_one_tile_after_longer_ones(long_tables, dim, wide):  # noqa: F811
    """Requests of three, two and one tile of 64 tokens in turn, several pairs to a thread block: the second stream of
    the tensor cores' kernel has no tile in the short ones. Against the oracle, then many times for equal bits."""
    import torch
    kvq, spec = base._mods()
    rng = np.random.default_rng(40 + dim)
    seq, trees = [150, 20, 100, 1] * 100, [5, 6, 7, 8] * 100
    base.check_tree(rng, 2, 4, dim, seq, trees, wide=wide)
    p = base.Pools(rng, 12, 2, dim, "e4m3", False)
    p.upload()
    table = torch.zeros((400, 256), dtype=torch.int32, device="cuda")
    table[:, :12] = dev(np.stack([rng.permutation(12) for _ in range(400)]).astype(np.int32))
    sees = base.random_sees(rng, trees)
    mask = spec.pack_tree_mask(dev(np.pad(sees, ((0, 0), (0, 64 - sees.shape[1]))))).contiguous()
    q = dev(rng.standard_normal((sum(trees), 8, dim)).astype(np.float16))
    lens, off = base.i32(seq), base.i32(np.concatenate([[0], np.cumsum(trees)]))
    ws = spec.tree_workspace(400, 2, 8, dim, 8)
    out = [torch.empty(q.shape, dtype=torch.float32 if wide else torch.float16, device="cuda") for _ in range(60)]
    for o in out:
        spec.fp8_tree_attention(q, *p.descs, table, lens, off, mask, 8, 4096, o, 0.0, ws)
    assert sum(not torch.equal(o, out[0]) for o in out) == 0


@pytest.mark.parametrize("gq,nodes", [(1, 3), (4, 6)])
def test_tree_behind_the_longest_context(gq, nodes):
    """A table of 2^27 - 1 blocks, all the same one but the last: 2^31 - 16 tokens in all. Every context token of a
    row of that block weighs the same, so the sums have a closed form."""
    import torch
    kvq, spec = base._mods()
    rng = np.random.default_rng(43)
    blocks, dim = 2 ** 27 - 1, 64
    length = blocks * 16 - nodes
    p = base.Pools(rng, 3, 1, dim, "e4m3", False)
    p.upload()
    table = torch.ones((1, blocks), dtype=torch.int32, device="cuda")
    table[0, -1] = 2
    q = rng.standard_normal((nodes, gq, dim)).astype(np.float16)
    sees = np.tril(np.ones((nodes, nodes), bool))
    mask = spec.pack_tree_mask(dev(np.pad(sees, ((0, 0), (0, 64 - nodes))))).contiguous()
    out = torch.zeros((nodes, gq, dim), dtype=torch.float32, device="cuda")
    ws = spec.tree_workspace(1, 1, gq, dim, nodes)
    spec.fp8_tree_attention(dev(q), *p.descs, table, base.i32([length]), base.i32([0, nodes]), mask, nodes, blocks * 16, out,
                            0.0, ws)
    got = out.cpu().numpy()
    assert int(ws[:4].view(torch.int32).item()) == 0
    kk, vv = (base.fp8.decode(p.nat[r][1:, 0].reshape(32, dim), "e4m3") * np.float64(p.scale[r][0]) for r in range(2))
    for i in range(nodes):
        count = np.concatenate([np.full(16, blocks - 1.0), np.ones(16 - nodes), sees[i]])
        for g in range(gq):
            s = kk @ q[i, g].astype(np.float64) / np.sqrt(dim)
            w = count * np.exp(s - s.max())
            # A sum is carried through at most 2^27 / 152 / 4 = 221 thousand steps in 32 bits by one thread and four
            # products a step: each may lose 2^-23 of it, the weights' sum and the outputs each for itself.
            bound = 2 * 4 * 221e3 * 2.0 ** -23 * (w @ np.abs(vv)) / w.sum()
            assert np.all(np.abs(got[i, g] - w @ vv / w.sum()) <= bound)
