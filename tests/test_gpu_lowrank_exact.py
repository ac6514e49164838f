"""The adapters' product is held in 32 bits whatever the result's type: where it cancels the base, only the error of FP32 sums
is left, and an infinity keeps its sign.  Tolerances are test_gpu_lowrank's for FP32 results, with a bf16 rounding behind them."""
import numpy as np
import pytest
import torch
from test_gpu_lowrank import U, Case, _half_ulp, _mixed, ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [True, False])
@pytest.mark.parametrize("r", [16, 48, 64, 128])
@pytest.mark.parametrize("m,n", [(1, 200), (40, 200), (40, 33), (300, 200), (300, 33), (4200, 136)])
def test_a_base_that_cancels(ops, m, n, r, int8):  # noqa: F811
    c = Case(m, n, 384, r, 3, _mixed(m, 3, r), seed=5, int8=int8, base="none")
    y, _ = c.ref(3)
    g = torch.Generator().manual_seed(r)
    c.base = torch.from_numpy(-y).float() + torch.randn((m, n), generator=g) * 1e-3
    want, err = c.ref(3)
    got = c.call(ops)
    assert got.dtype == torch.bfloat16
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= err + _half_ulp(np.abs(want) + err))
    f32 = c.call(ops, out_f32=True)
    assert torch.equal(got, f32.to(torch.bfloat16))  # the same sums, rounded once


@pytest.mark.parametrize("r", [16, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("base,epilogue", [("bf16", "none"), ("f32", "residual")])
def test_long_chunks(ops, r, base, epilogue):  # noqa: F811
    """Rows and columns enough for a CTA to keep as many positions as shared memory holds."""
    m, n = 2700, 7680
    c = Case(m, n, 128, r, 4, _mixed(m, 4, r).sort().values, base=base, epilogue=epilogue)
    want, err = c.ref(3)
    got = c.call(ops).double().cpu().numpy()
    assert np.all(np.abs(got - want) <= err + _half_ulp(np.abs(want) + err))


@pytest.mark.parametrize("m", [3, 300, 4200])
@pytest.mark.parametrize("out_f32", [False, True])
def test_an_infinity_keeps_its_sign(ops, m, out_f32):  # noqa: F811
    c = Case(m, 40, 128, 16, 1, [0] * m, int8=False, base="none", alpha=False)
    c.a[:], c.b[:] = 1.0, 1.0
    for value in (-np.inf, np.inf):
        c.x[1, 3] = value
        y = c.call(ops, out_f32=out_f32).float().cpu()
        assert bool((y[1] == value).all())
        assert torch.isfinite(y[[0, 2]]).all() and torch.isfinite(y[3:]).all()
    c.x[1, 4] = -np.inf
    assert torch.isnan(c.call(ops, out_f32=out_f32)[1]).all()
