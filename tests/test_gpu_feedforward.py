"""Feed-forward operators on the GPU against their definitions in 64 bits: add + RMS norm + INT8, W4A8 of few rows,
W4A8 grouped by expert.

Tolerances, all derived (u = 2^-24, one FP32 rounding):
  products   a group's integer sum is exact; G groups are scaled and added in FP32 in some order, then multiplied by the
             row's scale: at most (G + 12) roundings of partial sums that never exceed S = s_m sum_g |s_w acc_g|.
             The epilogue's GELU adds 4e-7 |g| + its slope (below 1.13) times that, the residual one rounding.
  norm       the sum of squares is K positive terms, summed in at most 64 + 16 steps a thread and a tree: 1 + 100 u of
             it, half of that in the root.  A rotated element is log2 b sums on top of the weight's rounding, none
             larger than its block's L1 norm.
  codes      |q s - z| <= s / 2 but for those errors.
  bf16       half a unit in the last place.
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


def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def _half_ulp_bf16(v):
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - 8)


# ---------------------------------------------------------- add + norm + INT8 --

def _sylvester(b):
    h = np.ones((1, 1))
    while h.shape[0] < b:
        h = np.block([[h, h], [h, -h]])
    return h


def _norm_ref(x, r, w, eps, b):
    """(z, bound on a computed z's error) in float64 from bf16-valued float32 inputs."""
    h = x.astype(np.float64) + (0.0 if r is None else r.astype(np.float64))
    rinv = 1.0 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    v = h * (1.0 if w is None else w.astype(np.float64))
    m, k = v.shape
    if b:
        z = (v.reshape(m, k // b, b) @ _sylvester(b)).reshape(m, k) / np.sqrt(b)
        l1 = np.repeat(np.abs(v).reshape(m, k // b, b).sum(2), b, 1) / np.sqrt(b)
    else:
        z, l1 = v, np.abs(v)
    steps = 4 + (int(np.log2(b)) if b else 0)
    return z * rinv, rinv * (steps * U * l1 + 60 * U * np.abs(z))


def _check_norm(a, h, x, r, w, eps, b):
    z, err = _norm_ref(x, r, w, eps, b)
    q = a.i8_codes.cpu().numpy().astype(np.float64)
    s = a.row_scale.cpu().numpy().astype(np.float64)
    top = np.abs(z).max(1)
    assert np.all(np.abs(s * 127 - top) <= err.max(1) + 4 * U * top), "row scale"
    assert np.all(np.abs(q) <= 127)
    assert np.all(np.abs(q * s[:, None] - z) <= s[:, None] * (0.5 + 127 * 8 * U) + 2 * err.max(1, keepdims=True)), "codes"
    assert np.all(np.abs(q).max(1)[top > 0] == 127)
    if r is not None:
        want = (torch.from_numpy(x) + torch.from_numpy(r)).to(torch.bfloat16)
        assert torch.equal(h.cpu().view(torch.int16), want.view(torch.int16)), "sum"


def _norm_inputs(m, k, seed, residual=True, weight=True):
    g = np.random.default_rng(seed)
    x = g.laplace(size=(m, k)).astype(np.float32)
    x[:, g.random(k) < 0.005] *= 50
    x = _bf16(x).float().numpy()
    r = _bf16(g.normal(size=(m, k))).float().numpy() if residual else None
    w = (g.random(k).astype(np.float32) + 0.5) if weight else None
    return x, r, w


def _norm_call(ops, x, r, w, eps, b, **kw):
    return ops.add_rmsnorm_quant(_bf16(x).cuda(), None if r is None else _bf16(r).cuda(),
                                 None if w is None else torch.from_numpy(w).cuda(), eps=eps, had_block=b, **kw)


@pytest.mark.parametrize("b", [0, 16, 64, 256])
@pytest.mark.parametrize("m,k", [(1, 256), (3, 512), (37, 768), (200, 1280), (5, 4096), (17, 4352), (9, 8448),
                                 (2, 16640), (3, 33024)])
def test_norm_shapes(ops, m, k, b):
    x, r, w = _norm_inputs(m, k, 100 * b + k + m)
    a, h = _norm_call(ops, x, r, w, 1e-6, b)
    _check_norm(a, h, x, r, w, 1e-6, b)


@pytest.mark.parametrize("m,k,b", [(1, 128, 64), (33, 384, 16), (130, 1920, 64), (65, 640, 0), (7, 12288, 64)])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", [False, True])
def test_norm_optional_operands(ops, m, k, b, residual, weight):
    x, r, w = _norm_inputs(m, k, m + k, residual, weight)
    a, h = _norm_call(ops, x, r, w, 1e-5, b)
    _check_norm(a, h, x, r, w, 1e-5, b)


@pytest.mark.parametrize("k", [256, 1920, 12288, 33024])
def test_norm_special_rows(ops, k):
    b = 64
    x, r, w = _norm_inputs(12, k, k)
    x[1], r[1] = 0, 0                        # padding
    x[2], r[2] = 0, 0
    x[2, k - 1] = 3.0                        # one-hot
    x[4, 5] = np.inf
    r[5, k - 3] = np.nan
    x[6, 0], r[6, 0] = np.inf, -np.inf
    x[7], r[7] = _bf16(x[7] * 1e-36).float().numpy(), 0   # eps alone; the largest value below 1e-30
    x[8, :], r[8, :] = 3e38, 0               # the sum of squares overflows
    x[9], r[9] = -x[9] - 0.0, 0
    a, h = _norm_call(ops, x, r, w, 1e-6, b)
    s, q = a.row_scale.cpu().numpy(), a.i8_codes.cpu().numpy()
    assert s[1] == 0 and not q[1].any()
    for bad in (4, 5, 6, 8):
        assert np.isnan(s[bad]) and not q[bad].any()
    fine = [i for i in range(12) if i not in (4, 5, 6, 8)]
    rows = torch.tensor(fine)
    part = type("A", (), dict(i8_codes=a.i8_codes.cpu()[rows], row_scale=a.row_scale.cpu()[rows]))
    _check_norm(part, h.cpu()[rows], x[fine], r[fine], w, 1e-6, b)


@pytest.mark.parametrize("k", [256, 1920, 33024])
def test_norm_in_place_and_alignment(ops, k):
    m, b = 19, 64
    x, r, w = _norm_inputs(m, k, 3 * k)
    want, hw = _norm_call(ops, x, r, w, 1e-6, b)
    for which in ("x", "residual"):
        xd, rd = _bf16(x).cuda(), _bf16(r).cuda()
        t = xd if which == "x" else rd
        a, h = ops.add_rmsnorm_quant(xd, rd, torch.from_numpy(w).cuda(), had_block=b, sum_out=t)
        assert h is t and torch.equal(h, hw)
        assert torch.equal(a.i8_codes, want.i8_codes) and torch.equal(a.row_scale, want.row_scale)

    def at16(v):  # 16-byte but not 32-byte aligned
        buf = torch.empty(v.numel() + 8, dtype=v.dtype, device="cuda")
        o = buf[8:].view(v.shape)
        o.copy_(v)
        assert o.data_ptr() % 32 == 16
        return o

    a, h = ops.add_rmsnorm_quant(at16(_bf16(x)), at16(_bf16(r)), torch.from_numpy(w).cuda(), had_block=b)
    assert torch.equal(h, hw) and torch.equal(a.i8_codes, want.i8_codes) and torch.equal(a.row_scale, want.row_scale)


def test_norm_beyond_32_bit_offsets(ops):
    m, k = 1_130_000, 1920  # 2.17e9 elements
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    r = torch.zeros_like(x)
    xs, rs, w = _norm_inputs(3, k, 5)
    rows = torch.tensor([0, m // 2 + 1, m - 1])
    x[rows.cuda()], r[rows.cuda()] = _bf16(xs).cuda(), _bf16(rs).cuda()
    a, h = ops.add_rmsnorm_quant(x, r, torch.from_numpy(w).cuda(), had_block=64, sum_out=r)
    part = type("A", (), dict(i8_codes=a.i8_codes[rows.cuda()], row_scale=a.row_scale[rows.cuda()]))
    _check_norm(part, h[rows.cuda()], xs, rs, w, 1e-6, 64)
    assert int((a.row_scale != 0).sum()) == 3


def test_norm_feeds_the_gemm(ops):
    """The codes are sixbit_hadamard_quant's operand: INT8 qgemm and qgemv of them agree."""
    x, r, w = _norm_inputs(24, 1920, 8)
    a, _ = _norm_call(ops, x, r, w, 1e-6, 64)
    g = torch.Generator().manual_seed(1)
    pw = ops.pack_weights((torch.randn((272, 1920), generator=g) * 0.02).cuda(), 64)
    y, v = ops.qgemm(a, None, pw, ops.MODE_INT8, out_f32=True), ops.qgemv(a, pw, out_f32=True)
    q, s = a.i8_codes.double(), a.row_scale.double()
    bound = (q.abs() @ torch.full((272, 1920), 7.0, dtype=torch.float64, device="cuda").mT) * s[:, None]
    assert torch.all((y.double() - v.double()).abs() <= 64 * U * bound * float(pw.i4_scales.max()))


# ------------------------------------------------------------------- products --

def _unpack(w4):
    w = w4.astype(np.int16)
    q = np.stack((w & 15, w >> 4), -1).reshape(*w4.shape[:-1], -1)
    return (q ^ 8) - 8


def _weights(g, lead, n, k):
    q = g.integers(-7, 8, size=lead + (n, k)).astype(np.int8)
    u = (q & 15).astype(np.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), (g.random(lead + (k // 128, n)) * 0.02 + 0.001).astype(np.float32)


def _rows(g, m, k):
    return (g.integers(-127, 128, size=(m, k)).astype(np.int8), (g.random(m) * 0.05 + 0.01).astype(np.float32))


def _product(q, s, w4, ws, epi, res):
    """(reference, tolerance before the output's rounding) of one weight, float64."""
    m, k = q.shape
    n, gr = w4.shape[0], k // 128
    w = _unpack(w4).astype(np.float64).reshape(n, gr, 128)
    acc = np.einsum("mgk,ngk->gmn", q.astype(np.float64).reshape(m, gr, 128), w, optimize=True)
    t = acc * ws.astype(np.float64)[:, None, :]
    y = t.sum(0) * s.astype(np.float64)[:, None]
    tol = (gr + 12) * U * np.abs(t).sum(0) * s[:, None]
    if epi == 1:
        y = 0.5 * y * erfc(-y / np.sqrt(2.0))
        tol = 1.13 * tol + 4e-7 * np.abs(y) + 1e-30
    elif epi == 2:
        y = y + res.astype(np.float64)
        tol = tol + U * np.abs(y)
    return y, tol + 1e-37


def _check_product(y, ref, tol):
    f32 = y.dtype == torch.float32
    y = y.float().cpu().numpy().astype(np.float64)
    lim = tol if f32 else tol + _half_ulp_bf16(np.abs(ref) + tol)
    bad = np.abs(y - ref) > lim
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3], y[bad][:3], ref[bad][:3])


def _epi_args(g, epi, m, n):
    res = _bf16(g.normal(size=(m, n))) if epi == 2 else None
    return res, (None if res is None else res.cuda()), (None if res is None else res.float().numpy())


@pytest.mark.parametrize("m", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 24, 31, 32])
@pytest.mark.parametrize("n,k", [(1, 128), (17, 256), (130, 1024), (257, 1920), (48, 7680)])
def test_qgemv_shapes(ops, m, n, k):
    g = np.random.default_rng(m * 1000 + n + k)
    q, s = _rows(g, m, k)
    w4, ws = _weights(g, (), n, k)
    epi = (m + n) % 3
    res, rd, rn = _epi_args(g, epi, m, n)
    f32 = (m + k // 128) % 2 == 0
    y = ops.qgemv(ops.int8_act(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()),
                  ops.Int4Weights(torch.from_numpy(w4).cuda(), torch.from_numpy(ws).cuda()), epilogue=epi,
                  residual=rd, out_f32=f32)
    assert y.dtype == (torch.float32 if f32 else torch.bfloat16)
    _check_product(y, *_product(q, s, w4, ws, epi, rn))


@pytest.mark.parametrize("m", [1, 4, 6, 12, 32])
@pytest.mark.parametrize("n,k", [(1111, 640), (3072, 12288), (7680, 1920), (15361, 384)])
def test_qgemv_model_shapes(ops, m, n, k):
    g = np.random.default_rng(m + n)
    q, s = _rows(g, m, k)
    w4, ws = _weights(g, (), n, k)
    res, rd, rn = _epi_args(g, 2, m, n)
    y = ops.qgemv(ops.int8_act(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()),
                  ops.Int4Weights(torch.from_numpy(w4).cuda(), torch.from_numpy(ws).cuda()), epilogue=2, residual=rd,
                  out=rd)  # in place on the residual
    assert y is rd
    _check_product(y, *_product(q, s, w4, ws, 2, rn))


@pytest.mark.parametrize("m", [1, 4, 5, 16, 32])
def test_qgemv_extreme_codes(ops, m):
    """Every product at its largest (the group sum 128 * 889 and, with a -8 nibble, 130048) and a NaN row scale."""
    n, k = 40, 512
    q = np.full((m, k), 127, np.int8)
    q[:, 1::2] = -127
    s = np.ones(m, np.float32)
    s[m - 1] = np.nan
    w4 = np.full((n, k // 2), (9 << 4) | 7, np.uint8)  # 7 at even k, -7 at odd k
    w4[1] = (7 << 4) | 8                               # -8, 7
    ws = np.ones((k // 128, n), np.float32)
    y = ops.qgemv(ops.int8_act(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()),
                  ops.Int4Weights(torch.from_numpy(w4).cuda(), torch.from_numpy(ws).cuda()), out_f32=True).cpu().numpy()
    want = q.astype(np.int64) @ _unpack(w4).astype(np.int64).T
    assert np.array_equal(y[:m - 1], want[:m - 1].astype(np.float32)) and np.isnan(y[m - 1]).all()


def _grouped(ops, g, offsets, m, n, k, epi=0, f32=False, fill=None, err=None, **kw):
    e = len(offsets) - 1
    q, s = _rows(g, m, k)
    w4, ws = _weights(g, (e,), n, k)
    res, rd, rn = _epi_args(g, epi, m, n)
    out = torch.full((m, n), 777.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    y = ops.qgemm_grouped(ops.int8_act(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()),
                          ops.Int4Weights(torch.from_numpy(w4).cuda(), torch.from_numpy(ws).cuda()),
                          torch.tensor(offsets, dtype=torch.int32, device="cuda"), epilogue=epi, residual=rd, out=out,
                          err=err, **kw)
    assert y is out
    valid = [(a, b) if 0 <= a <= b <= m else (0, 0) for a, b in zip(offsets, offsets[1:])]
    owners = np.zeros(m, int)
    for a, b in valid:
        owners[a:b] += 1
    for i, (a, b) in enumerate(valid):
        rows = np.arange(a, b)[owners[a:b] == 1]  # a row that two experts claim (bad offsets) holds either's
        if len(rows):
            _check_product(y[torch.from_numpy(rows).cuda()],
                           *_product(q[rows], s[rows], w4[i], ws[i], epi, None if rn is None else rn[rows]))
    assert torch.all(y[torch.from_numpy(owners == 0).cuda()] == 777.0)


@pytest.mark.parametrize("counts", [[1], [5], [0, 1, 0], [3, 0, 0, 9, 1], [32], [33], [64, 65], [130, 0, 1, 31],
                                    [16] * 8, [0] * 7 + [1], [200, 1, 191, 193], [385, 0, 576]])
@pytest.mark.parametrize("n,k", [(16, 128), (129, 384), (300, 1920)])
def test_grouped_ragged(ops, counts, n, k):
    g = np.random.default_rng(sum(counts) * 7 + n + k)
    offsets = [0] + list(np.cumsum(counts))
    epi = (sum(counts) + n) % 3
    _grouped(ops, g, [int(o) for o in offsets], offsets[-1], n, k, epi, f32=(n + len(counts)) % 2 == 0)


@pytest.mark.parametrize("epi", [0, 1, 2])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n", [128, 251, 1000])
def test_grouped_epilogues(ops, epi, f32, n):
    g = np.random.default_rng(n + epi)
    _grouped(ops, g, [0, 7, 7, 300, 420], 420, n, 640, epi, f32)


@pytest.mark.parametrize("counts", [[3, 20], [90, 40], [300, 217]])
def test_grouped_extreme_codes(ops, counts):
    """Every code with every nibble, and group sums at their largest: exact integers in a float32 output."""
    n, k, m = 160, 512, sum(counts)
    q = np.full((m, k), 127, np.int8)
    q[1::3] = -127
    q[2::3] = (np.arange(k) % 255 - 127).astype(np.int8)
    q[::7, 1::2] *= -1
    w4 = np.empty((2, n, k // 2), np.uint8)
    w4[0] = (9 << 4) | 7                                                    # 7 at even k, -7 at odd k
    w4[0, 1] = (7 << 4) | 8                                                 # -8, 7
    w4[1] = ((np.arange(n)[:, None] + np.arange(k // 2)[None]) % 256).astype(np.uint8)
    ws = np.ones((2, k // 128, n), np.float32)
    offsets = [0, counts[0], m]
    y = ops.qgemm_grouped(ops.int8_act(torch.from_numpy(q).cuda(), torch.ones(m, device="cuda")),
                          ops.Int4Weights(torch.from_numpy(w4).cuda(), torch.from_numpy(ws).cuda()),
                          torch.tensor(offsets, dtype=torch.int32, device="cuda"), out_f32=True).cpu().numpy()
    for e in range(2):
        r = slice(offsets[e], offsets[e + 1])
        assert np.array_equal(y[r], (q[r].astype(np.int64) @ _unpack(w4[e]).astype(np.int64).T).astype(np.float32))


@pytest.mark.parametrize("counts", [[8], [9], [15, 1], [16, 17], [31, 33], [47], [48], [95, 96, 97], [128, 64, 63],
                                    [1] * 17, [0] * 40 + [4], [2, 0, 14] * 6])
@pytest.mark.parametrize("n,k", [(130, 640), (64, 1152)])
def test_grouped_every_form_and_tile_end(ops, counts, n, k):
    """Row counts on both sides of each form's limits and of each copied box, with a part of a batch at the end of K."""
    g = np.random.default_rng(sum(counts) + 3 * n + k)
    offsets = [0] + [int(o) for o in np.cumsum(counts)]
    _grouped(ops, g, offsets, offsets[-1], n, k, (len(counts) + n) % 3, f32=n == 64)


@pytest.mark.parametrize("counts", [[1, 4], [16, 5], [17, 30], [40, 2, 9], [96, 97], [150, 31]])
@pytest.mark.parametrize("code,nibble", [(127, 7), (127, -8), (-128, 7), (-128, -8), (None, None)])
def test_grouped_sums_at_their_limits(ops, counts, code, nibble):
    """Codes and weights all at one end, or at either end by chance: exact integers in a float32 output."""
    g = np.random.default_rng(11)
    n, k, m, e = 136, 384, sum(counts), len(counts)
    q = np.full((m, k), code, np.int8) if code is not None else (g.integers(0, 2, (m, k)) * 255 - 128).astype(np.int8)
    v = np.full((e, n, k), nibble) if nibble is not None else g.integers(0, 2, (e, n, k)) * 15 - 8
    w4 = ((v[..., 0::2] & 15) | ((v[..., 1::2] & 15) << 4)).astype(np.uint8)
    offsets = [0] + [int(o) for o in np.cumsum(counts)]
    y = ops.qgemm_grouped(ops.int8_act(torch.from_numpy(q).cuda(), torch.ones(m, device="cuda")),
                          ops.Int4Weights(torch.from_numpy(w4).cuda(), torch.ones(e, k // 128, n, device="cuda")),
                          torch.tensor(offsets, dtype=torch.int32, device="cuda"), out_f32=True).cpu().numpy()
    for i in range(e):
        r = slice(offsets[i], offsets[i + 1])
        assert np.array_equal(y[r], (q[r].astype(np.int64) @ v[i].T).astype(np.float32))


@pytest.mark.parametrize("m", [16, 17, 25, 32])
@pytest.mark.parametrize("code,nibble", [(127, -8), (-128, -8), (None, None)])
def test_qgemv_many_outputs(ops, m, code, nibble):
    """More weight rows than two tiles of 16 for each of two CTAs an SM, an odd number: exact integers."""
    g = np.random.default_rng(m)
    n, k = 64 * torch.cuda.get_device_properties(0).multi_processor_count + 21, 384
    q = np.full((m, k), code, np.int8) if code is not None else (g.integers(0, 2, (m, k)) * 255 - 128).astype(np.int8)
    v = np.full((n, k), nibble) if nibble is not None else g.integers(0, 2, (n, k)) * 15 - 8
    w4 = ((v[:, 0::2] & 15) | ((v[:, 1::2] & 15) << 4)).astype(np.uint8)
    y = ops.qgemv(ops.int8_act(torch.from_numpy(q).cuda(), torch.ones(m, device="cuda")),
                  ops.Int4Weights(torch.from_numpy(w4).cuda(), torch.ones(k // 128, n, device="cuda")),
                  out_f32=True).cpu().numpy()
    assert np.array_equal(y, (q.astype(np.int64) @ v.T).astype(np.float32))


def test_grouped_many_experts(ops):
    g = np.random.default_rng(5)
    counts = g.integers(0, 4, size=300)
    offsets = [0] + [int(v) for v in np.cumsum(counts)]
    _grouped(ops, g, offsets, offsets[-1], 72, 256, 1)


def test_grouped_gaps_are_left_alone(ops):
    g = np.random.default_rng(6)
    _grouped(ops, g, [3, 10, 10, 41], 60, 130, 256)
    _grouped(ops, g, [100, 250, 500], 600, 130, 256)


def test_grouped_bad_offsets_are_reported(ops):
    g = np.random.default_rng(7)
    for offsets, m in (([0, 20, 10, 40], 40), ([0, 10, 50], 40), ([-5, 10, 40], 40), ([0, 300, 200, 400], 400),
                       ([0, 2 ** 31 - 1, 40], 40)):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        _grouped(ops, g, offsets, m, 64, 256, err=err)
        assert err.item() == 7
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    _grouped(ops, g, [0, 10, 40], 40, 64, 256, err=err)
    assert err.item() == 0


def test_grouped_beyond_32_bit_offsets(ops):
    """Weights of more than 2^31 bytes and activations of more than 2^31 codes."""
    k, n, e, m = 12288, 7680, 48, 60
    g = torch.Generator(device="cuda").manual_seed(3)
    codes = torch.randint(0, 256, (e, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    assert codes.numel() > 2 ** 31
    scales = torch.rand((e, k // 128, n), generator=g, device="cuda") * 0.01
    q = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    s = torch.rand(m, generator=g, device="cuda")
    offsets = [0] * (e - 1) + [20, m]
    y = ops.qgemm_grouped(ops.int8_act(q, s), ops.Int4Weights(codes, scales),
                          torch.tensor(offsets, dtype=torch.int32, device="cuda"), out_f32=True)
    for i in (e - 2, e - 1):
        a, b = offsets[i], offsets[i + 1]
        pick = slice(n - 64, n)
        _check_product(y[a:b, pick], *_product(q[a:b].cpu().numpy(), s[a:b].cpu().numpy(), codes[i, pick].cpu().numpy(),
                                               scales[i, :, pick].cpu().numpy(), 0, None))
    del codes, scales, y
    m, n = 180_000, 32
    codes = torch.randint(0, 256, (2, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.rand((2, k // 128, n), generator=g, device="cuda") * 0.01
    q = torch.randint(-127, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    assert q.numel() > 2 ** 31
    s = torch.rand(m, generator=g, device="cuda")
    y = ops.qgemm_grouped(ops.int8_act(q, s), ops.Int4Weights(codes, scales),
                          torch.tensor([0, 90_001, m], dtype=torch.int32, device="cuda"), out_f32=True)
    for rows, i in ((slice(89_900, 90_001), 0), (slice(90_001, 90_050), 1), (slice(m - 70, m), 1)):
        _check_product(y[rows], *_product(q[rows].cpu().numpy(), s[rows].cpu().numpy(), codes[i].cpu().numpy(),
                                          scales[i].cpu().numpy(), 0, None))


def test_pack_experts_matches_the_dense_layer(ops):
    """Experts packed from float weights give what each layer's own qgemm gives."""
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.randn((3, 144, 384), generator=g, device="cuda") * 0.02
    x = torch.randn((70, 384), generator=g, device="cuda").to(torch.bfloat16)
    a = ops.hadamard_quant(x, 64, ops.MODE_INT8)
    offsets = [0, 20, 20, 70]
    y = ops.qgemm_grouped(a, ops.pack_experts(w, 64), torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                          out_f32=True)
    for e in range(3):
        d = ops.qgemm(a, None, ops.pack_weights(w[e], 64), ops.MODE_INT8, out_f32=True)
        rows = slice(offsets[e], offsets[e + 1])
        bound = a.i8_codes.double().abs().sum(1, keepdim=True) * a.row_scale.double()[:, None] * 7 * 0.02
        assert torch.all((y[rows].double() - d[rows].double()).abs() <= 32 * U * bound[rows])


# ------------------------------------------------------- streams, graphs, modes --

def _all_three(ops, x, r, w, wd, we, offsets, **kw):
    a, h = ops.add_rmsnorm_quant(x, r, w, had_block=64, **kw)
    return ops.qgemv(a, wd, epilogue=ops.EPI_GELU, **kw), ops.qgemm_grouped(a, we, offsets, **kw), h


def _setup(ops, m=24, k=640, n=320):
    g = np.random.default_rng(11)
    x, r, w = _norm_inputs(m, k, 12)
    wd, we = _weights(g, (), n, k), _weights(g, (3,), n, k)
    dev = lambda t: ops.Int4Weights(*(torch.from_numpy(v).cuda() for v in t))  # noqa: E731
    return (_bf16(x).cuda(), _bf16(r).cuda(), torch.from_numpy(w).cuda(), dev(wd), dev(we),
            torch.tensor([0, 5, 5, m], dtype=torch.int32, device="cuda"))


def test_side_stream_and_repeatability(ops):
    args = _setup(ops)
    want = [t.clone() for t in _all_three(ops, *args)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = _all_three(ops, *args, stream=side)
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    with torch.cuda.stream(side):
        got = _all_three(ops, *args)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_cuda_graph(ops):
    args = _setup(ops)
    want = [t.clone() for t in _all_three(ops, *args)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _all_three(ops, *args)
    x = args[0].clone()
    args[0].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(got[2], want[2])
    args[0].copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_offsets_change_between_replays(ops):
    """The row counts live on the device: a captured product follows them."""
    x, r, w, _, we, offsets = _setup(ops)
    a, _ = ops.add_rmsnorm_quant(x, r, w, had_block=64)
    torch.cuda.synchronize()
    out = torch.empty((24, we.n), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.qgemm_grouped(a, we, offsets, out=out)
    for o in ([0, 24, 24, 24], [0, 0, 11, 24], [0, 1, 2, 24]):
        offsets.copy_(torch.tensor(o, dtype=torch.int32))
        graph.replay()
        want = ops.qgemm_grouped(a, we, torch.tensor(o, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_grouped_in_a_switched_branch(ops):
    """The product in a body of a device-selected branch of a captured graph, beside work outside of it."""
    x, r, w, _, we, offsets = _setup(ops)
    a, _ = ops.add_rmsnorm_quant(x, r, w, had_block=64)
    want = ops.qgemm_grouped(a, we, offsets)
    out = torch.zeros_like(want)
    ws = torch.empty(ops.qgemm_grouped_workspace_bytes(a.m, a.k), dtype=torch.uint8, device="cuda")
    word = torch.tensor([ops.MODE_INT8], dtype=torch.int32, device="cuda")
    stream, body = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        sw = ops.GraphSwitch(stream, body, word, ops.MODE_INT8, 1)
        with sw.branch(0):
            ops.qgemm_grouped(a, we, offsets, out=out, ws=ws)
        sw.close()
    for mode, runs in ((ops.MODE_INT8, True), (ops.MODE_BF16, False), (ops.MODE_INT8, True)):
        word.fill_(mode)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want if runs else torch.zeros_like(want))


def test_mode_word(ops):
    x, r, w, wd, we, offsets = _setup(ops)
    want = _all_three(ops, x, r, w, wd, we, offsets)
    for mode, runs in ((ops.MODE_INT8 | 1 << 10, True), (ops.MODE_NVFP4, False), (ops.MODE_BF16, False),
                       (ops.MODE_SKIP, False)):
        word = torch.tensor([mode], dtype=torch.int32, device="cuda")
        h = torch.full_like(x, 3.0)
        out = ops.int8_act(torch.full(x.shape, 5, dtype=torch.int8, device="cuda"),
                           torch.full((x.shape[0],), 2.0, device="cuda"))
        ops.add_rmsnorm_quant(x, r, w, had_block=64, out=out, sum_out=h, mode_dev=word)
        a, _ = ops.add_rmsnorm_quant(x, r, w, had_block=64)
        v, e = torch.full_like(want[0], 9.0), torch.full_like(want[1], 9.0)
        ops.qgemv(a, wd, epilogue=ops.EPI_GELU, out=v, mode_dev=word)
        ops.qgemm_grouped(a, we, offsets, out=e, mode_dev=word)
        if runs:
            assert torch.equal(v, want[0]) and torch.equal(e, want[1]) and torch.equal(h, want[2])
            assert torch.equal(out.i8_codes, a.i8_codes)
        else:
            assert torch.all(v == 9) and torch.all(e == 9) and torch.all(h == 3)
            assert torch.all(out.i8_codes == 5) and torch.all(out.row_scale == 2)


def test_no_rows(ops):
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    a, h = ops.add_rmsnorm_quant(x, x.clone(), had_block=16)
    assert a.i8_codes.shape == (0, 256) and h.shape == (0, 256)
    g = np.random.default_rng(1)
    w = ops.Int4Weights(*(torch.from_numpy(v).cuda() for v in _weights(g, (), 40, 256)))
    assert ops.qgemv(a, w).shape == (0, 40)
    we = ops.Int4Weights(*(torch.from_numpy(v).cuda() for v in _weights(g, (2,), 40, 256)))
    assert ops.qgemm_grouped(a, we, torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 40)


def test_refusals(ops):
    x, r, w, wd, we, offsets = _setup(ops)
    a, _ = ops.add_rmsnorm_quant(x, r, w, had_block=64)
    before = ops.launch_count()
    bad = [
        lambda: ops.add_rmsnorm_quant(x.float(), r, w),
        lambda: ops.add_rmsnorm_quant(x, r[:-1], w),
        lambda: ops.add_rmsnorm_quant(x, r, w.double()),
        lambda: ops.add_rmsnorm_quant(x, r, w[1:]),
        lambda: ops.add_rmsnorm_quant(x[:, ::2], None, None),
        lambda: ops.add_rmsnorm_quant(x, None, None, sum_out=r),
        lambda: ops.add_rmsnorm_quant(x.cpu(), None, None),
        lambda: ops.qgemv(ops.int8_act(a.i8_codes[:, :-128].contiguous(), a.row_scale), wd),
        lambda: ops.qgemv(ops.int8_act(a.i8_codes, a.row_scale[1:]), wd),
        lambda: ops.qgemv(a, we),
        lambda: ops.qgemv(a, wd, residual=torch.empty((24, wd.n), dtype=torch.bfloat16, device="cuda")),
        lambda: ops.qgemv(a, wd, out=torch.empty((24, wd.n), dtype=torch.float16, device="cuda")),
        lambda: ops.qgemm_grouped(a, wd, offsets),
        lambda: ops.qgemm_grouped(a, we, offsets[:-1]),
        lambda: ops.qgemm_grouped(a, we, offsets.long()),
        lambda: ops.qgemm_grouped(a, we, offsets, ws=torch.empty(8, dtype=torch.uint8, device="cuda")),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    status = [
        lambda: ops.add_rmsnorm_quant(x, r, w, eps=0.0),
        lambda: ops.add_rmsnorm_quant(x, r, w, eps=float("nan")),
        lambda: ops.add_rmsnorm_quant(x, r, w, had_block=32),
        lambda: ops.add_rmsnorm_quant(x, r, w, had_block=256),      # 640 % 256
        lambda: ops.qgemv(ops.int8_act(a.i8_codes.repeat(2, 1), a.row_scale.repeat(2)), wd),   # 48 rows
        lambda: ops.qgemv(a, wd, epilogue=3),
        lambda: ops.qgemv(a, wd, epilogue=ops.EPI_RESIDUAL),
        lambda: ops.qgemm_grouped(a, we, offsets, epilogue=ops.EPI_RESIDUAL),
    ]
    from video_dit_mixed_gb300.abi import SixbitError
    for f in status:
        with pytest.raises(SixbitError):
            f()
    assert ops.launch_count() == before
