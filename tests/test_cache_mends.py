"""CPU checks of the cache's and the attention's calls that once went wrong."""

import pytest

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------ strides

@pytest.mark.parametrize("stride", [1, 64, 127, 128, 129, 1001])
def test_the_stride_of_one_row_says_nothing(q4lib, stride):
    t = torch.zeros(2048, dtype=torch.float16).as_strided((1, 2, 64), (stride, 64, 1))
    assert q4lib._row_stride(t, "q", 2, 64) == 128
    assert q4lib._row_stride(torch.zeros(5, 300).as_strided((2, 2, 64), (300, 64, 1)), "q", 2, 64) == 300


# ------------------------------------------------------------------ sizes

@pytest.mark.parametrize("tokens", [1 << 63, 1 << 70, -(1 << 70)])
@pytest.mark.parametrize("with_offsets", [False, True])
def test_more_rows_than_64_bits_hold(q4lib, tokens, with_offsets):
    """The native way leaves such a call to the full one, which refuses it (here for its host tensors)."""
    c = torch.zeros((4, 2, 2, 1, 9 * 64), dtype=torch.uint8)
    tables, lengths = torch.zeros(3, 2, dtype=torch.int32), torch.ones(3, dtype=torch.int32)
    offsets = torch.arange(4, dtype=torch.int32) if with_offsets else None
    with pytest.raises(ValueError, match="device tensor"):
        q4lib.q4_cache_read(c, tables, lengths, offsets, tokens=tokens)
