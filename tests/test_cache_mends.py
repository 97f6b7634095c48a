"""CPU checks of the cache's and the attention's calls that once went wrong."""

import shutil
import subprocess
from pathlib import Path

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


# ------------------------------------------------------------------ positions

@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_windows_of_rows_far_before_the_first_position(tmp_path):
    """The kernels' rule of what a row sees, compiled for the host with its overflows trapped: rows
    of a sequence with up to 2^31 - 2 rows more than positions."""
    text = (Path(__file__).resolve().parent.parent / "bit_block_quantized_q4_amd" / "csrc" / "q4_cache.hpp").read_text()
    at = text.index("__device__ __forceinline__ void seen_by(")
    rule = text[at:text.index("\n}\n", at) + 3]
    (tmp_path / "rule.cpp").write_text("""
#include <cstdio>
#include <cstdint>
#include <initializer_list>
#define __device__
#define __forceinline__ inline
struct Attention { int causal, window; };
""" + rule + """
int main() {
  const int most = 1 << 30;
  for (int causal = 0; causal < 2; ++causal)
    for (int window : {0, 1, 2, 100, most - 1, most})
      for (int length : {0, 1, 100, most})
        for (int64_t p : {-2147483647ll, -2147483646ll, -1073741825ll, -1073741824ll, -101ll, -1ll, 0ll, 99ll,
                          static_cast<long long>(most) - 1}) {
          if (p >= length) continue;
          int lo, hi;
          seen_by(Attention{causal, window}, length, static_cast<int>(p), &lo, &hi);
          const int64_t to = causal ? (p + 1 < 0 ? 0 : p + 1) : length, after = window ? p - window + 1 : 0;
          const int64_t from = after < 0 ? 0 : after;
          if (hi != to || lo != (from < to ? from : to)) {
            std::printf("causal %d window %d length %d position %lld: %d .. %d\\n", causal, window, length,
                        static_cast<long long>(p), lo, hi);
            return 1;
          }
        }
  return 0;
}
""")
    build = ["g++", "-std=c++17", "-O2", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
             str(tmp_path / "rule.cpp"), "-o", str(tmp_path / "rule")]
    subprocess.run(build, check=True)
    run = subprocess.run([str(tmp_path / "rule")], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout + run.stderr
