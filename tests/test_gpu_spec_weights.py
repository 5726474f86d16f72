"""Tree attention of few rows holds its softmax weights as exactly as the single-token decode, whatever the output's type."""
import numpy as np
import pytest

import test_gpu_spec as base
from kvq_helpers import dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,fmt,hq", [(128, "e4m3", 16), (64, "e5m2", 2), (64, "e4m3", 8)])
def test_tree_of_one_node_with_fp16_output_is_the_decode_rounded(dim, fmt, hq):
    """The decode with fp32 output is a few 1e-6 from the 64-bit result on values of unit size, and so is the tree before
    its output is rounded: what remains is half a step of fp16. One fp16 weight a token (2^-12 relative on average)
    would move outputs near 0 by several times that."""
    import torch
    kvq, spec = base._mods()
    rng = np.random.default_rng(60 + dim + hq)
    b, h = 3, 2
    p = base.Pools(rng, 40, h, dim, fmt, False)
    p.upload()
    table = rng.permutation(36).reshape(3, 12).astype(np.int32)
    lens = [150, 1, 77]
    q = rng.standard_normal((b, hq, dim)).astype(np.float16)
    got, _ = base.run_tree(spec, p, table, [n - 1 for n in lens], [1, 1, 1], np.ones((3, 1), bool), q, False)
    out = torch.empty((b, hq, dim), dtype=torch.float32, device="cuda")
    n = kvq.fp8_decode_workspace_bytes(b, hq, dim)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    kvq.fp8_decode_attention(dev(q), *p.descs, dev(table), base.i32(lens), b, hq, 12, 192, out, True, 0.0, ws, n)
    want = host(out).astype(np.float64)
    assert np.all(np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 2e-5)
