"""The grouped product's bounded waits, run out on purpose (nothing faults): with sixbit_debug_gemm_timeout every CTA's
token producer withholds its first slot and the limit is 20 ms, so the kernel must record SIXBIT_ETIMEOUT, stop its
roles, free its tensor memory and return; the next launch on the same context must be right."""
import ctypes as C

import pytest
import torch

pytestmark = pytest.mark.gpu
ETIMEOUT = 6


@pytest.mark.parametrize("rows", [40, 300])  # token tiles of 32 and of 128
def test_wait_timeout_is_reported_and_the_context_recovers(rows):
    from video_dit_mixed_gb300 import abi, ops
    lib = abi.lib()
    e, n, k = 2, 300, 1024
    g = torch.Generator(device="cuda").manual_seed(3)
    a = ops.int8_act(torch.randint(-127, 128, (rows, k), generator=g, device="cuda", dtype=torch.int8),
                     torch.rand(rows, generator=g, device="cuda"))
    w = ops.Int4Weights(torch.randint(0, 256, (e, n, k // 2), generator=g, device="cuda", dtype=torch.uint8),
                        torch.rand((e, k // 128, n), generator=g, device="cuda"))
    offsets = torch.tensor([0, rows // 3, rows], dtype=torch.int32, device="cuda")
    want = ops.qgemm_grouped(a, w, offsets)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream = C.c_void_p(torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert lib.sixbit_debug_gemm_timeout(20_000_000, 1) == 0
    try:
        ops.qgemm_grouped(a, w, offsets, err=err)
        status = lib.sixbit_check(C.c_void_p(err.data_ptr()), stream)
    finally:
        assert lib.sixbit_debug_gemm_timeout(0, 0) == 0
    assert status == ETIMEOUT, lib.sixbit_status_str(status)
    got = ops.qgemm_grouped(a, w, offsets, err=err)
    assert lib.sixbit_check(C.c_void_p(err.data_ptr()), stream) == 0
    assert torch.equal(got, want)
