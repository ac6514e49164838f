"""The experts' weighted sum against 64 bits: k products and k sums of FP32, none above S = sum_j |w d|, so 2 k 2^-24 S, and
half a step of the output's type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _half_ulp(v):
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - 8)


def _inputs(t, k, h, r, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    d = torch.randn((r, h), generator=g).to(dtype)
    rows = torch.randint(0, r, (t, k), generator=g, dtype=torch.int32)
    return d, rows, torch.rand((t, k), generator=g)


def _check(y, d, rows, w):
    dd, ww, rr = d.double().numpy(), w.double().numpy(), rows.numpy()
    terms = np.where(rr[..., None] >= 0, dd[np.maximum(rr, 0)] * ww[..., None], 0.0)
    ref, bound = terms.sum(1), 2 * rr.shape[1] * U * np.abs(terms).sum(1)
    if y.dtype == torch.bfloat16:
        bound = bound + _half_ulp(np.abs(ref) + bound)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= bound)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("out_f32", [False, True])
@pytest.mark.parametrize("t,k,h", [(1, 1, 8), (1, 2, 1920), (7, 3, 250), (5, 32, 129), (64, 5, 2056), (300, 8, 640),
                                   (1000, 2, 1920), (2, 4, 30001)])
def test_sum(ops, t, k, h, dtype, out_f32):
    d, rows, w = _inputs(t, k, h, max(1, t * k - 1), dtype, t + k + h)
    rows[t // 2, 0] = -1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.moe_combine(d.cuda(), rows.cuda(), w.cuda(), out_f32=out_f32, err=err)
    assert y.dtype == (torch.float32 if out_f32 else torch.bfloat16)
    _check(y, d, rows, w)
    ops.check_err(err, "sum")


@pytest.mark.parametrize("h", [256, 250])
def test_rows_out_of_range_are_reported(ops, h):
    d, rows, w = _inputs(9, 3, h, 11, torch.float32, 1)
    rows[4, 1], rows[6, 2] = 11, -2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.moe_combine(d.cuda(), rows.cuda(), w.cuda(), err=err)
    with pytest.raises(RuntimeError):
        ops.check_err(err, "sum")
    rows[4, 1], rows[6, 2] = -1, -1
    _check(y, d, rows, w)


def test_not_finite_values_stay_in_their_tokens(ops):
    d, rows, w = _inputs(6, 2, 64, 12, torch.float32, 2)
    rows[:] = torch.arange(12, dtype=torch.int32).view(6, 2)
    d[3, 5], d[8, 7] = float("nan"), float("inf")
    y = ops.moe_combine(d.cuda(), rows.cuda(), w.cuda()).float().cpu()
    assert torch.isnan(y[1, 5]) and torch.isinf(y[4, 7])
    y[1, 5] = y[4, 7] = 0
    assert torch.isfinite(y).all()


def test_alignment_output_and_stream(ops):
    d, rows, w = _inputs(33, 2, 128, 66, torch.bfloat16, 3)
    dv, rv, wv = d.cuda(), rows.cuda(), w.cuda()
    want = ops.moe_combine(dv, rv, wv)
    buf = torch.empty(66 * 128 + 1, dtype=torch.bfloat16, device="cuda")
    odd = buf[1:].view(66, 128)
    odd.copy_(dv)
    assert torch.equal(ops.moe_combine(odd, rv, wv), want)
    obuf = torch.full((33 * 128 + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = obuf[1:-2].view(33, 128)
    assert ops.moe_combine(dv, rv, wv, out=out) is out and torch.equal(out, want)
    assert obuf[0] == 7 and bool((obuf[-2:] == 7).all())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = ops.moe_combine(dv, rv, wv, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.moe_combine(dv, rv, wv)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_beyond_32_bit_offsets(ops):
    r, h = 1_130_000, 1920
    d = torch.zeros((r, h), dtype=torch.bfloat16, device="cuda")
    d[r - 1], d[r // 2] = 2.0, 3.0
    rows = torch.tensor([[r - 1, r // 2], [0, r - 1]], dtype=torch.int32, device="cuda")
    y = ops.moe_combine(d, rows, torch.tensor([[0.5, 1.0], [1.0, 0.25]], device="cuda"))
    assert bool((y[0] == 4).all()) and bool((y[1] == 0.5).all())


def test_empty_and_refusals(ops):
    d = torch.zeros((4, 64), device="cuda")
    rows, w = torch.zeros((3, 2), dtype=torch.int32, device="cuda"), torch.zeros((3, 2), device="cuda")
    assert ops.moe_combine(d, rows[:0], w[:0]).shape == (0, 64)
    none = torch.empty((0, 64), device="cuda")
    assert not ops.moe_combine(none, torch.full_like(rows, -1), w).any()
    for bad in (lambda: ops.moe_combine(d.cpu(), rows, w), lambda: ops.moe_combine(d.half(), rows, w),
                lambda: ops.moe_combine(d, rows.long(), w), lambda: ops.moe_combine(d, rows, w[:2]),
                lambda: ops.moe_combine(d, rows[0], w), lambda: ops.moe_combine(d[:, ::2], rows, w),
                lambda: ops.moe_combine(d, rows, w, out=d)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(RuntimeError):
        ops.moe_combine(d, torch.zeros((1, 33), dtype=torch.int32, device="cuda"), torch.zeros((1, 33), device="cuda"))
