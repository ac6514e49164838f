"""A token that is not a number stays one, and changes no other token: through the INT8 quantization (its scale, as the
oracle's) and through whole feed-forward layers."""
import numpy as np
import pytest
import torch

from oracle import quant

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


# every kernel form: half blocks a lane (b 64), register rows, two passes (K beyond 16384)
@pytest.mark.parametrize("b,k", [(64, 128), (64, 1920), (64, 7680), (64, 12288), (64, 16512), (16, 256), (16, 1920),
                                 (16, 16640), (256, 512), (256, 7680), (256, 16640)])
def test_int8_scale_of_rows_that_hold_a_nan(ops, b, k):
    m = 37
    g = np.random.default_rng(b + k)
    x = torch.from_numpy(g.normal(size=(m, k)).astype(np.float32)).to(torch.bfloat16)
    clean = ops.hadamard_quant(x.cuda(), b, ops.MODE_INT8)
    bad = {0: 0, 3: k - 1, 9: k // 2, 20: min(k - 1, 1100), 36: 17}
    for row, col in bad.items():
        x[row, col] = NAN
    x[30, 5], x[30, 6] = INF, -INF              # an infinity less an infinity
    a = ops.hadamard_quant(x.cuda(), b, ops.MODE_INT8)
    s = a.row_scale.cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = quant.hadamard_quant(x.float().numpy(), b, "int8")["s"]
    assert np.array_equal(np.isnan(s), np.isnan(want)) and set(np.flatnonzero(np.isnan(s))) == set(bad) | {30}
    fine = torch.from_numpy(~np.isnan(s)).cuda()
    assert torch.equal(a.i8_codes[fine], clean.i8_codes[fine]) and torch.equal(a.row_scale[fine], clean.row_scale[fine])


@pytest.mark.parametrize("kind", ["dense", "experts"])
@pytest.mark.parametrize("t", [1, 4, 20, 300])
@pytest.mark.parametrize("value", [NAN, INF, -INF, 3e38])
def test_layers(ops, kind, t, value):
    """(3e38: a finite token whose sum of squares overflows FP32 has a NaN scale)"""
    from video_dit_mixed_gb300 import ffn
    hid, f, e = 256, 640, 4
    g = torch.Generator(device="cuda").manual_seed(t)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if kind == "dense":
        layer = ffn.FFN(*(ops.pack_weights(rand(*s) * 0.05, 64) for s in ((f, hid), (hid, f))))
    else:
        layer = ffn.MoEFFN(rand(e, hid), *(ops.pack_experts(rand(e, *s) * 0.05, 64) for s in ((f, hid), (hid, f))), top_k=2)
    x, r = rand(t, hid).to(torch.bfloat16), rand(t, hid).to(torch.bfloat16)
    y0, h0 = layer(x, r)
    x = x.clone()
    x[t // 2, 7] = value
    y, h = layer(x, r)
    layer.check()
    others = torch.arange(t, device="cuda") != t // 2
    assert bool(y[t // 2].isnan().all())
    assert torch.equal(y[others], y0[others]) and torch.equal(h[others], h0[others])
