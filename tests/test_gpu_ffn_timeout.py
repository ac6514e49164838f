"""A bounded wait that runs out inside a feed-forward layer is reported by layer.check().  The waits are made to run out
with sixbit_debug_gemm_timeout (a withheld first copy, limit 20 ms): nothing faults, and the next call is right."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind,t", [("dense", 300), ("experts", 40), ("experts", 300)])
def test_layer_reports_a_wait_that_ran_out(kind, t):
    from video_dit_mixed_gb300 import abi, ffn, ops
    lib = abi.lib()
    hid, f, e = 256, 640, 3
    g = torch.Generator(device="cuda").manual_seed(t)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if kind == "dense":
        layer = ffn.FFN(*(ops.pack_weights(rand(*s) * 0.05, 64) for s in ((f, hid), (hid, f))))
    else:
        layer = ffn.MoEFFN(rand(e, hid), *(ops.pack_experts(rand(e, *s) * 0.05, 64) for s in ((f, hid), (hid, f))), top_k=2)
    x, r = rand(t, hid).to(torch.bfloat16), rand(t, hid).to(torch.bfloat16)
    want = layer(x, r)
    layer.check()
    assert lib.sixbit_debug_gemm_timeout(20_000_000, 1) == 0
    try:
        layer(x, r)
        with pytest.raises(abi.SixbitError, match=type(layer).__name__):
            layer.check()
    finally:
        assert lib.sixbit_debug_gemm_timeout(0, 0) == 0
    got = layer(x, r)
    layer.check()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(x, r)
    layer.check(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
