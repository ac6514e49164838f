"""Feed-forward operators at the far ends of their arguments, on the GPU.  References and tolerances are those of
test_gpu_feedforward."""
import gc

import numpy as np
import pytest
import torch

from test_gpu_feedforward import _bf16, _check_product, _product

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def test_grouped_rows_of_two_gigabytes(ops):
    """N = 2^30: two rows of a bf16 Y are 2^32 bytes apart.  Y on the residual's place; the weights are zero but for some
    columns, so that any value at a wrong place shows."""
    n, k, m = 1 << 30, 128, 9
    gc.collect()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 110 * 2 ** 30:
        pytest.skip("needs 110 GiB of device memory")
    g = np.random.default_rng(1)
    q, s = g.integers(-127, 128, size=(m, k)).astype(np.int8), (g.random(m) * 0.05 + 0.01).astype(np.float32)
    codes = torch.zeros((1, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.ones((1, 1, n), dtype=torch.float32, device="cuda")
    y = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    picks = []
    for at in (0, 1 << 20, (1 << 29) - 17, n - 150):
        pick = slice(at, at + 150)
        w4 = g.integers(0, 256, size=(150, k // 2)).astype(np.uint8)
        ws = (g.random((1, 150)) * 0.02 + 0.001).astype(np.float32)
        res = _bf16(g.normal(size=(m, 150)))
        codes[0, pick], scales[0, :, pick], y[:, pick] = (torch.from_numpy(w4).cuda(), torch.from_numpy(ws).cuda(),
                                                          res.cuda())
        picks.append((pick, w4, ws, res.float().numpy()))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = ops.qgemm_grouped(ops.int8_act(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()),
                            ops.Int4Weights(codes, scales), torch.tensor([0, m], dtype=torch.int32, device="cuda"),
                            epilogue=ops.EPI_RESIDUAL, residual=y, out=y, err=err)
    assert out is y and err.item() == 0
    for pick, w4, ws, res in picks:
        _check_product(y[:, pick], *_product(q, s, w4, ws, 2, res))
        y[:, pick] = 0
    for row in y:
        assert not bool(row.any())


@pytest.mark.parametrize("m,e", [(7, 15), (40, 65), (300, 3), (300, 1023)])
def test_grouped_offsets_that_claim_every_row_many_times(ops, m, e):
    """0, M, 0, M, ...: reported; with one weight for all experts, every row has its result all the same."""
    n, k = 136, 384
    g = np.random.default_rng(m)
    q, s = g.integers(-127, 128, size=(m, k)).astype(np.int8), (g.random(m) * 0.05 + 0.01).astype(np.float32)
    w4 = g.integers(0, 256, size=(n, k // 2)).astype(np.uint8)
    ws = (g.random((k // 128, n)) * 0.02 + 0.001).astype(np.float32)
    w = ops.Int4Weights(torch.from_numpy(w4).cuda().expand(e, -1, -1).contiguous(),
                        torch.from_numpy(ws).cuda().expand(e, -1, -1).contiguous())
    offsets = torch.tensor([0 if i % 2 == 0 else m for i in range(e + 1)], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.qgemm_grouped(ops.int8_act(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()), w, offsets, out_f32=True,
                          err=err)
    assert err.item() == 7
    _check_product(y, *_product(q, s, w4, ws, 0, None))
