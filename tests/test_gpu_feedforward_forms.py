"""Every form of the grouped product (dot products, narrow and wide token tiles) through side streams, captured graphs,
device-selected branches and the mode word, in place on the residual, and on pointers with the least alignment that is
accepted.  References and tolerances are those of test_gpu_feedforward."""
import numpy as np
import pytest
import torch

from test_gpu_feedforward import _bf16, _check_product, _product, _rows, _weights

pytestmark = pytest.mark.gpu
FORMS = [7, 24, 200]  # rows over three experts: dot products, token tiles of 32 and of 96


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


class Case:
    def __init__(self, ops, m, n=320, k=640, e=3, seed=11):
        g = np.random.default_rng(seed + m)
        self.m, self.n, self.k = m, n, k
        self.q, self.s = _rows(g, m, k)
        self.w4, self.ws = _weights(g, (e,), n, k)
        self.res = _bf16(g.normal(size=(m, n)))
        self.bounds = [0, m // 3, m // 3, m]
        self.a = ops.int8_act(torch.from_numpy(self.q).cuda(), torch.from_numpy(self.s).cuda())
        self.w = ops.Int4Weights(torch.from_numpy(self.w4).cuda(), torch.from_numpy(self.ws).cuda())
        self.one = ops.Int4Weights(self.w.i4_codes[0], self.w.i4_scales[0])
        self.offsets = torch.tensor(self.bounds, dtype=torch.int32, device="cuda")

    def check(self, y, epi, bounds=None, one=False):
        res = self.res.float().numpy()
        bounds = bounds or self.bounds
        for i, (a, b) in enumerate(zip(bounds, bounds[1:]) if not one else [(0, self.m)]):
            if b > a:
                _check_product(y[a:b], *_product(self.q[a:b], self.s[a:b], self.w4[i], self.ws[i], epi, res[a:b]))


@pytest.mark.parametrize("m", FORMS)
@pytest.mark.parametrize("f32", [False, True])
def test_residual_in_place(ops, m, f32):
    c = Case(ops, m)
    y = c.res.cuda()
    if f32:  # (a float32 output has no bf16 residual's place)
        out = ops.qgemm_grouped(c.a, c.w, c.offsets, ops.EPI_RESIDUAL, residual=y, out_f32=True)
    else:
        out = ops.qgemm_grouped(c.a, c.w, c.offsets, ops.EPI_RESIDUAL, residual=y, out=y)
        assert out is y
    c.check(out, 2)


def _shifted(t, by):
    """t's values at an address `by` elements past a 16-byte boundary, guarded on both sides."""
    buf = torch.full((t.numel() + 64,), 7.0, dtype=t.dtype, device="cuda")
    o = buf[16 + by:16 + by + t.numel()].view(t.shape)
    o.copy_(t)
    return buf, o


@pytest.mark.parametrize("m", FORMS)
@pytest.mark.parametrize("n", [320, 129])
@pytest.mark.parametrize("epi", [0, 1, 2])
@pytest.mark.parametrize("by,res_by", [(1, 1), (1, 2), (2, 1), (0, 1)])
def test_grouped_pointers_of_least_alignment(ops, m, n, epi, by, res_by):
    """Y and the residual 2-byte (by 1) or 4-byte (by 2) aligned, N even and odd."""
    c = Case(ops, m, n=n)
    buf, y = _shifted(torch.zeros((m, n), dtype=torch.bfloat16), by)
    _, r = _shifted(c.res, res_by)
    assert y.data_ptr() % 4 == 2 * (by & 1) and r.data_ptr() % 4 == 2 * (res_by & 1)
    ops.qgemm_grouped(c.a, c.w, c.offsets, epi, residual=r if epi == 2 else None, out=y)
    c.check(y, epi)
    flat = buf.float()
    assert bool((flat[:16 + by] == 7).all()) and bool((flat[16 + by + m * n:] == 7).all())


@pytest.mark.parametrize("m", [1, 2, 5, 12, 32])
@pytest.mark.parametrize("n", [320, 129])
@pytest.mark.parametrize("epi,f32", [(0, True), (1, False), (2, False)])
def test_qgemv_pointers_of_least_alignment(ops, m, n, epi, f32):
    c = Case(ops, m, n=n)
    buf, y = _shifted(torch.zeros((m, n), dtype=torch.float32 if f32 else torch.bfloat16), 1)
    _, r = _shifted(c.res, 1)
    ops.qgemv(c.a, c.one, epi, residual=r if epi == 2 else None, out=y)
    c.check(y, epi, one=True)
    flat = buf.float()
    assert bool((flat[:17] == 7).all()) and bool((flat[17 + m * n:] == 7).all())


@pytest.mark.parametrize("m", FORMS)
@pytest.mark.parametrize("epi", [0, 1, 2])
def test_side_stream(ops, m, epi):
    c = Case(ops, m)
    r = c.res.cuda() if epi == 2 else None
    want = ops.qgemm_grouped(c.a, c.w, c.offsets, epi, residual=r)
    c.check(want, epi)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    got = [ops.qgemm_grouped(c.a, c.w, c.offsets, epi, residual=r, stream=side[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got)


@pytest.mark.parametrize("m", FORMS)
def test_graph_follows_its_inputs(ops, m):
    """A captured product reads codes and offsets at each replay (digits and product start together in it)."""
    c = Case(ops, m)
    out = torch.empty((m, c.n), dtype=torch.bfloat16, device="cuda")
    ops.qgemm_grouped(c.a, c.w, c.offsets, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.qgemm_grouped(c.a, c.w, c.offsets, out=out)
    g = np.random.default_rng(3)
    for bounds in ([0, 0, 0, m], [0, m, m, m], [0, 1, m - 1, m]):
        c.q, c.s = _rows(g, m, c.k)
        c.a.i8_codes.copy_(torch.from_numpy(c.q))
        c.a.row_scale.copy_(torch.from_numpy(c.s))
        c.offsets.copy_(torch.tensor(bounds, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, 0, bounds)


@pytest.mark.parametrize("m", FORMS)
def test_mode_word_and_switched_branch(ops, m):
    c = Case(ops, m)
    want = ops.qgemm_grouped(c.a, c.w, c.offsets)
    c.check(want, 0)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for mode in (ops.MODE_INT8, ops.MODE_NVFP4, ops.MODE_BF16, ops.MODE_SKIP, ops.MODE_INT8 | 1 << 10):
        word.fill_(mode)
        y = torch.full_like(want, 9.0)
        for _ in range(3):
            ops.qgemm_grouped(c.a, c.w, c.offsets, out=y, mode_dev=word)
        assert torch.equal(y, want) if mode & 0xFF == ops.MODE_INT8 else bool((y == 9).all())
    out = torch.zeros_like(want)
    ws = torch.empty(ops.qgemm_grouped_workspace_bytes(m, c.k), dtype=torch.uint8, device="cuda")
    stream, body = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sw = ops.GraphSwitch(stream, body, word, ops.MODE_INT8, 1)
        with sw.branch(0):
            ops.qgemm_grouped(c.a, c.w, c.offsets, out=out, ws=ws)
        sw.close()
    for mode in (ops.MODE_INT8, ops.MODE_BF16, ops.MODE_INT8):
        word.fill_(mode)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want if mode == ops.MODE_INT8 else torch.zeros_like(want))
