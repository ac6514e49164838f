"""A copy of the gated norm that does not arrive in time is reported, and the next launch is right (the wait is shortened
and each warp's first copy withheld; nothing faults)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [256, 1920, 4096, 7680])
def test_timeout_is_reported(k):
    from video_dit_mixed_gb300 import abi, ops
    m = 1500
    g = torch.Generator(device="cuda").manual_seed(k)
    x, r = (torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.rand(k, generator=g, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        return ops.gated_rmsnorm_quant(x, r, w, w, w, had_block=64, err=err)

    want, h = call()
    ops.check_err(err, "norm")
    try:
        abi.check(abi.lib().sixbit_debug_gemm_timeout(20_000_000, 1), "debug")
        call()
        with pytest.raises(abi.SixbitError, match="time"):
            ops.check_err(err, "norm")
    finally:
        abi.check(abi.lib().sixbit_debug_gemm_timeout(0, 0), "debug")
    a, h2 = call()
    ops.check_err(err, "norm")
    assert torch.equal(a.i8_codes, want.i8_codes) and torch.equal(a.row_scale, want.row_scale) and torch.equal(h, h2)
