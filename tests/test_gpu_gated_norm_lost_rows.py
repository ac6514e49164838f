"""Rows of the gated norm whose copy did not arrive in time are NaN, not what shared memory held (the wait is shortened and
each warp's first copy withheld; nothing faults)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [256, 1920, 4096, 7680])
@pytest.mark.parametrize("post", [False, True])
def test_lost_rows_are_nan(k, post):
    from video_dit_mixed_gb300 import abi, ops
    m = 1500
    g = torch.Generator(device="cuda").manual_seed(k)
    x, r = (torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand(k, generator=g, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(quantize):
        return ops.gated_rmsnorm_quant(x, r, w, w if post else None, w, had_block=64 if quantize else 0, quantize=quantize,
                                       err=err)

    call(True), call(False)
    try:
        abi.check(abi.lib().sixbit_debug_gemm_timeout(20_000_000, 1), "debug")
        for quantize in (True, False):
            a, h = call(quantize)
            with pytest.raises(abi.SixbitError, match="time"):
                ops.check_err(err, "norm")
            assert torch.isnan(h).all()
            if quantize:
                assert torch.isnan(a.row_scale).all() and not a.i8_codes.any()
            else:
                assert torch.isnan(a).all()
    finally:
        abi.check(abi.lib().sixbit_debug_gemm_timeout(0, 0), "debug")
    a, h = call(True)
    ops.check_err(err, "norm")
    assert torch.isfinite(a.row_scale).all() and torch.isfinite(h).all()
