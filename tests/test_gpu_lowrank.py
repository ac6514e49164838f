"""Low-rank adapters beside a projection, against 64 bits.

Tolerances (u = 2^-24): an MMA adds 16 exact products to its sum and may drop two units of the largest of them, so a sum
of K products is off by at most (K / 16 + 20) 4 u S, S = sum |x a| (20: the warps' and CTAs' sums, the row's scale and
alpha).  The product with B takes A x to 2^-16 of itself (2^-24 for FP32 results), carries its error, and adds
(R / 16 parts + 20) 4 u of its own terms.  Base and residual are one rounding each, GELU has a slope below 1.13 and is
right to 4e-7 |g|, and the output is half a step.
"""
import numpy as np
import pytest
import torch
from scipy.special import erfc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _half_ulp(v):
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - 8)


class Case:
    def __init__(self, m, n, k, r, count, ids, seed=0, int8=True, alpha=True, base="f32", epilogue="none"):
        g = torch.Generator().manual_seed(seed + m + n + k + r)

        def randn(*s):
            return torch.randn(s, generator=g)

        self.a = (randn(count, r, k) * k ** -0.5).to(torch.bfloat16)
        self.b = randn(count, n, r).to(torch.bfloat16)
        self.alpha = torch.rand(count, generator=g) + 0.5 if alpha else None
        if int8:
            self.codes = torch.randint(-128, 128, (m, k), generator=g).to(torch.int8)
            self.scale = torch.rand(m, generator=g) * 0.03 + 0.005
            self.x64 = self.codes.double() * self.scale.double()[:, None]
        else:
            self.codes = None
            self.x = randn(m, k).to(torch.bfloat16)
            self.x64 = self.x.double()
        self.ids = ids if isinstance(ids, torch.Tensor) else torch.tensor(ids, dtype=torch.int32)
        self.base = {"f32": randn(m, n), "bf16": randn(m, n).to(torch.bfloat16), "none": None}[base]
        self.res = randn(m, n).to(torch.bfloat16) if epilogue == "residual" else None
        self.epilogue = epilogue
        self.m, self.n, self.k, self.r, self.count = m, n, k, r, count

    def call(self, ops, **kw):
        def dev(t):
            return None if t is None else t.cuda()

        x = ops.int8_act(self.codes.cuda(), self.scale.cuda()) if self.codes is not None else self.x.cuda()
        epi = {"none": ops.EPI_NONE, "gelu": ops.EPI_GELU, "residual": ops.EPI_RESIDUAL}[self.epilogue]
        args = dict(base=dev(self.base), epilogue=epi, residual=dev(self.res))
        args.update(kw)
        return ops.lowrank_add(x, ops.LowRank(self.a.cuda(), self.b.cuda(), dev(self.alpha)), dev(self.ids), **args)

    def ref(self, parts):
        """(result, its error before the output's rounding)"""
        x, m, n = self.x64.numpy(), self.m, self.n
        y, e = np.zeros((m, n)), np.zeros((m, n))
        for i in range(self.count):
            at = (self.ids == i).numpy().nonzero()[0]
            if len(at):
                a, b = self.a[i].double().numpy(), self.b[i].double().numpy()
                f = 1.0 if self.alpha is None else float(self.alpha[i])
                v, s = x[at] @ a.T * f, np.abs(x[at]) @ np.abs(a).T * f
                ev = (self.k / 16 + 20) * 4 * U * s
                y[at] = v @ b.T
                terms = (np.abs(v) + ev) @ np.abs(b).T
                e[at] = ev @ np.abs(b).T + (2.0 ** (-8 * parts) + (self.r / 16 * parts + 20) * 4 * U) * terms
        if self.base is not None:
            y = y + self.base.double().numpy()
            e = e + U * np.abs(y)
        if self.epilogue == "gelu":
            y = 0.5 * y * erfc(-y / np.sqrt(2))
            e = 1.13 * e + 4e-7 * np.abs(y) + 1e-7 * np.abs(y)
        elif self.epilogue == "residual":
            y = y + self.res.double().numpy()
            e = e + U * np.abs(y)
        return y, e

    def check(self, y):
        f32 = y.dtype == torch.float32
        want, err = self.ref(3 if f32 else 2)
        got = y.double().cpu().numpy()
        bound = err + (U * np.abs(want) if f32 else _half_ulp(np.abs(want) + err))
        if self.epilogue == "gelu":  # its negative tail is right to 2e-7 of the argument's size
            bound = bound + 2e-6
        assert np.all(np.abs(got - want) <= bound)


def _mixed(m, count, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-1, count, (m,), generator=g, dtype=torch.int32)


@pytest.mark.parametrize("m", [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 100, 127, 128, 129, 257, 300, 1000])
@pytest.mark.parametrize("int8", [True, False])
def test_rows(ops, m, int8):
    for count in (1, 5, 40):
        c = Case(m, 200, 256, 16, count, _mixed(m, count, m), int8=int8)
        c.check(c.call(ops))


@pytest.mark.parametrize("r", [16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("k", [128, 640, 1920])
def test_ranks_and_depths(ops, r, k):
    for m in (1, 40, 300):
        c = Case(m, 72, k, r, 3, _mixed(m, 3, r))
        c.check(c.call(ops))
        c.check(c.call(ops, out_f32=True))


@pytest.mark.parametrize("n", [1, 7, 8, 31, 32, 33, 250, 256, 257, 1111, 2048])
@pytest.mark.parametrize("epilogue", ["none", "gelu", "residual"])
def test_widths_and_epilogues(ops, n, epilogue):
    for m, base in ((1, "f32"), (37, "bf16"), (290, "none"), (290, "f32")):
        c = Case(m, n, 128, 32, 4, _mixed(m, 4, n), base=base, epilogue=epilogue, alpha=m != 37)
        c.check(c.call(ops))
        c.check(c.call(ops, out_f32=True))


@pytest.mark.parametrize("r", [16, 32, 48, 64, 96, 128])
@pytest.mark.parametrize("m,count", [(1535, 3), (1536, 1), (2500, 300), (4095, 2), (5001, 6)])
@pytest.mark.parametrize("int8", [True, False])
def test_many_rows(ops, m, count, r, int8):
    """Mixed rows, and the same rows with their requests side by side."""
    ids = _mixed(m, count, r)
    for order in (ids, ids.sort().values):
        c = Case(m, 136, 384, r, count, order, int8=int8, base="bf16")
        c.check(c.call(ops))
    c = Case(m, 33, 1920, r, count, ids, int8=int8)
    c.check(c.call(ops, out_f32=True))


@pytest.mark.parametrize("m", [32, 200, 1003, 4100])
def test_runs_of_requests(ops, m):
    ids = torch.full((m,), -1, dtype=torch.int32)
    cuts = [0, m // 7, m // 7 + 1, m // 2, m - 3, m]
    for i, (a, b) in enumerate(zip(cuts, cuts[1:])):
        ids[a:b] = (2, 0, -1, 3, 2)[i]
    c = Case(m, 320, 384, 64, 4, ids, base="bf16", epilogue="gelu")
    c.check(c.call(ops))


def test_as_many_adapters_as_there_may_be(ops):
    count, k, n = ops.MAX_ADAPTERS, 128, 8
    for m in (20, 700, 5000):
        g = torch.Generator().manual_seed(m)
        ids = torch.randint(0, count, (m,), generator=g, dtype=torch.int32)
        ids[:3] = torch.tensor([0, count - 1, -1], dtype=torch.int32)
        a = torch.zeros((count, 16, k), dtype=torch.bfloat16, device="cuda")
        a[:, 0, 0] = 1.0
        b = torch.zeros((count, n, 16), dtype=torch.bfloat16, device="cuda")
        b[:, :, 0] = (torch.arange(count, device="cuda") % 251).to(torch.bfloat16)[:, None]  # whole numbers below 256
        x = torch.ones((m, k), dtype=torch.bfloat16, device="cuda")
        y = ops.lowrank_add(x, ops.LowRank(a, b), ids.cuda(), out_f32=True)
        want = torch.where(ids >= 0, ids % 251, 0).float()
        assert torch.equal(y.cpu(), want[:, None].expand(m, n))
    with pytest.raises(RuntimeError):
        ops.lowrank_add(x, ops.LowRank(torch.zeros((count + 1, 16, k), dtype=torch.bfloat16, device="cuda"),
                                       torch.zeros((count + 1, n, 16), dtype=torch.bfloat16, device="cuda")), ids.cuda())


def test_every_row_its_own_adapter_and_one_for_all(ops):
    for ids in (torch.randperm(64, generator=torch.Generator().manual_seed(1)).int(), torch.full((64,), 9).int(),
                torch.full((64,), -1).int()):
        c = Case(64, 136, 7680, 16, 64, ids)
        c.check(c.call(ops))


def test_rows_without_an_adapter_are_the_base(ops):
    for m in (5, 300):
        c = Case(m, 64, 128, 16, 2, torch.full((m,), -1, dtype=torch.int32))
        assert torch.equal(c.call(ops).cpu(), c.base.to(torch.bfloat16))
        assert torch.equal(c.call(ops, out_f32=True).cpu(), c.base)


def test_numbers_out_of_range_are_reported(ops):
    for m in (9, 400):
        c = Case(m, 64, 128, 16, 3, _mixed(m, 3))
        c.ids[[2, 7]] = torch.tensor([3, -2], dtype=torch.int32)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        y = c.call(ops, err=err)
        with pytest.raises(RuntimeError):
            ops.check_err(err, "adapters")
        c.ids[[2, 7]] = -1
        c.check(y)


def test_not_finite_rows_stay_alone(ops):
    c = Case(40, 64, 128, 16, 2, _mixed(40, 2))
    c.ids[[5, 33]] = torch.tensor([1, 0], dtype=torch.int32)
    c.scale[5], c.scale[33] = float("nan"), float("inf")
    y = c.call(ops)
    assert torch.isnan(y[5].float()).all() and not torch.isfinite(y[33].float()).any()
    rest = [i for i in range(40) if i not in (5, 33)]
    assert torch.isfinite(y[rest].float()).all()
    c.scale[[5, 33]] = 0.01
    d = c.call(ops)
    assert torch.equal(d[rest], y[rest])
    x = Case(3, 8, 128, 16, 1, [0, 0, 0], int8=False, base="none", alpha=False)  # an infinity keeps its sign
    x.b[:], x.a[:] = 1.0, 0.0
    x.a[0, 0] = 1.0
    x.x[1, 3] = float("-inf")
    y = x.call(ops)
    assert torch.isinf(y[1]).all() and bool((y[1] < 0).all()) or torch.isnan(y[1]).all()
    assert torch.isfinite(y[[0, 2]].float()).all()


def test_in_place_alignment_streams_modes(ops):
    for m in (3, 300):
        c = Case(m, 96, 256, 32, 3, _mixed(m, 3), base="bf16")
        want = c.call(ops)
        base = c.base.cuda()
        assert c.call(ops, base=base, out=base) is base and torch.equal(base, want)
        f = Case(m, 96, 256, 32, 3, c.ids, base="f32")
        fw, fb = f.call(ops, out_f32=True), f.base.cuda()
        f.call(ops, base=fb, out=fb)
        assert torch.equal(fb, fw)
        res = Case(m, 96, 256, 32, 3, c.ids, epilogue="residual")
        rw, rb = res.call(ops), res.res.cuda()
        res.call(ops, residual=rb, out=rb)
        assert torch.equal(rb, rw)
        buf = torch.full((m * 96 + 3,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = buf[1:-2].view(m, 96)
        c.call(ops, out=out)
        assert torch.equal(out, want) and buf[0] == 7 and bool((buf[-2:] == 7).all())
        mode = torch.tensor([ops.MODE_NVFP4], dtype=torch.int32, device="cuda")
        out = torch.full((m, 96), 5.0, dtype=torch.bfloat16, device="cuda")
        c.call(ops, out=out, mode_dev=mode)
        assert bool((out == 5).all())
        mode.fill_(ops.MODE_INT8)
        c.call(ops, out=out, mode_dev=mode)
        assert torch.equal(out, want)
        ws = torch.full((ops.lowrank_workspace_bytes(m, 32),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(c.call(ops, ws=ws), want)


@pytest.mark.parametrize("m", [1, 20, 300, 4200])
def test_streams_and_graphs(ops, m):
    c = Case(m, 256, 1920, 16, 4, _mixed(m, 4, 3), epilogue="gelu")
    want = c.call(ops)
    x = ops.int8_act(c.codes.cuda(), c.scale.cuda())
    w, ids, base = ops.LowRank(c.a.cuda(), c.b.cuda(), c.alpha.cuda()), c.ids.cuda(), c.base.cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    ys = []
    for _ in range(10):
        ys.append(ops.lowrank_add(x, w, ids, base, ops.EPI_GELU))
        ys.append(ops.lowrank_add(x, w, ids, base, ops.EPI_GELU, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in ys)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ops.lowrank_add(x, w, ids, base, ops.EPI_GELU)
        z = ops.lowrank_add(x, w, ids, base, ops.EPI_GELU)
    for _ in range(2):
        y.zero_(), z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want)


@pytest.mark.parametrize("b,rank", [(0, 16), (16, 4), (64, 20), (256, 128)])
def test_packing(ops, b, rank):
    """Rotated codes times the packed adapter are x A^T of the unrotated ones (to the codes' and bf16's roundings)."""
    g = torch.Generator().manual_seed(rank)
    count, n, k, m = 2, 24, 512, 6
    a = (torch.randn((count, rank, k), generator=g) * k ** -0.5).to(torch.bfloat16)
    bb = torch.randn((count, n, rank), generator=g).to(torch.bfloat16)
    x = torch.randn((m, k), generator=g).to(torch.bfloat16)
    w = ops.pack_lowrank(a.cuda(), bb.cuda(), None, b)
    assert w.rank == (rank + 15) // 16 * 16 and not w.a[:, rank:].any() and not w.b[:, :, rank:].any()
    ids = torch.tensor([0, 1, 0, 1, 1, 0], dtype=torch.int32)
    want = torch.stack([bb[i].double() @ (a[i].double() @ x[j].double()) for j, i in enumerate(ids.tolist())])
    if b:
        act = ops.hadamard_quant(x.cuda(), b, ops.MODE_INT8, out=ops.QActTensors(m, k, nvfp4=False))
    else:
        act = x.cuda()
    y = ops.lowrank_add(act, w, ids.cuda(), out_f32=True).double().cpu()
    # a code is off by half of the row's 1/127 (4 sigma of it here), A by 2^-9: together below 2% of the result's size
    assert float((y - want).norm() / want.norm()) < 0.03


def test_beyond_32_bit_offsets(ops):
    """Rows whose outputs lie beyond 2^31 elements, and adapters whose weights do."""
    m, n, k, r = 300_000, 7680, 128, 16
    x = torch.zeros((m, k), dtype=torch.int8, device="cuda")
    x[-1], x[m // 2] = 1, 2
    ids = torch.zeros(m, dtype=torch.int32, device="cuda")
    w = ops.LowRank(torch.ones((1, r, k), dtype=torch.bfloat16, device="cuda"),
                    torch.ones((1, n, r), dtype=torch.bfloat16, device="cuda"))
    y = ops.lowrank_add(ops.int8_act(x, torch.ones(m, device="cuda")), w, ids)
    assert bool((y[-1] == k * r).all()) and bool((y[m // 2] == 2 * k * r).all())
    assert int((y != 0).any(1).sum()) == 2
    del y, x
    count, n, r = 1200, 15360, 128  # 2.4e9 elements of B
    b = torch.zeros((count, n, r), dtype=torch.bfloat16, device="cuda")
    b[-1] = 1.0
    a = torch.zeros((count, r, k), dtype=torch.bfloat16, device="cuda")
    a[-1] = 1.0
    ids = torch.tensor([0, count - 1], dtype=torch.int32, device="cuda")
    y = ops.lowrank_add(torch.ones((2, k), dtype=torch.bfloat16, device="cuda"), ops.LowRank(a, b), ids)
    assert not y[0].any() and bool((y[1] == k * r).all())


def test_empty_and_refusals(ops):
    def z(*s, dtype=torch.bfloat16):
        return torch.zeros(s, dtype=dtype, device="cuda")

    w, ids = ops.LowRank(z(2, 16, 128), z(2, 40, 16), z(2, dtype=torch.float32)), z(3, dtype=torch.int32)
    x, act = z(3, 128), ops.int8_act(z(3, 128, dtype=torch.int8), z(3, dtype=torch.float32))
    assert ops.lowrank_add(x[:0], w, ids[:0]).shape == (0, 40)
    for bad in (lambda: ops.LowRank(z(2, 16, 128), z(2, 40, 32)), lambda: ops.LowRank(z(1, 16, 128), z(2, 40, 16)),
                lambda: ops.lowrank_add(x.cpu(), w, ids), lambda: ops.lowrank_add(x.float(), w, ids),
                lambda: ops.lowrank_add(z(3, 256), w, ids), lambda: ops.lowrank_add(x, w, ids.long()),
                lambda: ops.lowrank_add(x, w, ids[:2]), lambda: ops.lowrank_add(x, w, ids, z(3, 41)),
                lambda: ops.lowrank_add(act, w, ids, residual=z(3, 40)), lambda: ops.lowrank_add(act, w, ids, out=z(3, 48)),
                lambda: ops.lowrank_add(z(129, 128), w, z(129, dtype=torch.int32), ws=z(1, dtype=torch.uint8)),
                lambda: ops.pack_lowrank(z(2, 129, 128), z(2, 40, 129), None, 16),
                lambda: ops.lowrank_add(x, ops.LowRank(z(2, 16, 128), z(2, 40, 16), z(3, dtype=torch.float32)), ids)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.lowrank_add(x, w, ids, epilogue=ops.EPI_RESIDUAL), lambda: ops.lowrank_add(x, w, ids, epilogue=7),
                lambda: ops.lowrank_add(x, ops.LowRank(z(2, 8, 128), z(2, 40, 8)), ids),
                lambda: ops.lowrank_add(z(3, 64), ops.LowRank(z(2, 16, 64), z(2, 40, 16)), ids),
                lambda: ops.lowrank_add(x, ops.LowRank(z(2, 144, 128), z(2, 40, 144)), ids)):
        with pytest.raises(RuntimeError):
            bad()
