"""The W4A8 products' largest sizes at the C boundary (host only: nothing is enqueued)."""
import ctypes as C

import pytest

INT_MAX, ESHAPE = 2 ** 31 - 1, 2


@pytest.fixture(scope="module")
def lib():
    from video_dit_mixed_gb300 import abi
    return abi.lib(build_if_missing=True)


@pytest.mark.parametrize("n", [INT_MAX, INT_MAX - 31, INT_MAX - 127])
@pytest.mark.parametrize("m", [1, 2, 3, 20, 32])
def test_few_rows_refuse_widths_whose_last_tile_passes_32_bits(lib, n, m):
    from video_dit_mixed_gb300 import abi
    raw = C.create_string_buffer(4096)
    p = (C.addressof(raw) + 63) // 64 * 64
    qa, qw = abi.QAct(None, None, None, None, p, p, None), abi.Weights(None, None, None, None, p, p, None)
    before = lib.sixbit_launch_count()
    assert lib.sixbit_qgemv(C.byref(qa), C.byref(qw), m, n, 128, None, 0, None, p, None, None, None) == ESHAPE
    assert lib.sixbit_launch_count() == before


def test_grouped_tile_numbers_stay_in_32_bits(tmp_path):
    """Offsets that do not ascend (0, M, 0, M, ...) let every second of 1024 experts claim all rows: the device's count
    of tiles is capped before it becomes a tile number."""
    import os
    import shutil
    import subprocess
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = r"""
#include <cstdio>
#include "internal.h"
int main() {
  const int64_t grid = 152;
  int refused = 0;
  for (int tile : {32, 96})
    for (int64_t rows : {1ll, 96ll, 50000ll, 402653184ll, 805306368ll, 2147483647ll})
      for (int64_t n : {1ll, 128ll, 7680ll, 2097151ll, 2147483519ll})
        for (int experts : {1, 2, 7, 1024}) {
          if (sixbit::most_token_tiles(rows, tile, experts) > UINT32_MAX) {
            ++refused;
            continue;
          }
          int64_t claimed = 0;
          for (int e = 0; e < experts; e += 2) claimed += (rows + tile - 1) / tile;
          if (claimed > sixbit::most_token_tiles(rows, tile, experts)) return 1;  // (so below 2^32)
          const uint32_t tiles_n = static_cast<uint32_t>((n + 127) / 128);
          const int64_t all = sixbit::tile_count(static_cast<uint32_t>(claimed), tiles_n);
          // the next turn's number within unsigned 32 bits, nothing left out below the limit
          if (all > INT32_MAX || all + grid > UINT32_MAX) return 2;
          if (claimed * tiles_n <= INT32_MAX && all != claimed * tiles_n) return 3;
        }
  if (refused == 0) return 4;
  std::puts("ok");
}
"""
    src = tmp_path / "tiles.cc"
    src.write_text(code)
    exe = tmp_path / "tiles"
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    subprocess.run([cxx, "-std=c++17", "-I" + os.path.join(root, "include"), "-I" + os.path.join(cuda, "include"),
                    "-I" + os.path.join(root, "video_dit_mixed_gb300", "csrc"), str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"
