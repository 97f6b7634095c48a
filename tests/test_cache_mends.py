"""CPU checks of the cache's and the attention's calls that once went wrong."""

import pytest

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ strides

@pytest.mark.parametrize("stride", [1, 64, 127, 128, 129, 1001])
def test_the_stride_of_one_row_says_nothing(q4lib, stride):
    t = torch.zeros(2048, dtype=torch.float16).as_strided((1, 2, 64), (stride, 64, 1))
    assert q4lib._row_stride(t, "q", 2, 64) == 128
    assert q4lib._row_stride(torch.zeros(5, 300).as_strided((2, 2, 64), (300, 64, 1)), "q", 2, 64) == 300
