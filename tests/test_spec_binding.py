"""The speculative-decoding binding's reading of layouts, without a GPU."""
import pytest

spec = pytest.importorskip("quantized_kv_cache_quant_gb300.spec", reason="libkvq.so not built")


def test_one_row_has_no_stride_that_could_be_refused():
    """Rows may lie any multiple of 8 elements apart; a single one lies apart from nothing, whatever its tensor says."""
    import torch
    for stride in (1, 131, 1000):
        one = torch.empty_strided((1, 2, 64), (stride, 64, 1), dtype=torch.float16)
        assert spec._rows("k_new", one, 1, 2, 64, -1) == (one.data_ptr(), 128)
    two = torch.empty_strided((2, 2, 64), (136, 64, 1), dtype=torch.float16)
    assert spec._rows("k_new", two, 2, 2, 64, -1) == (two.data_ptr(), 136)
