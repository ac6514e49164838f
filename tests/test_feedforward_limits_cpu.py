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
