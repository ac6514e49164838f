"""Norms around a block's branch with gate, residual and modulation, against the definition in 64 bits.

Tolerances (u = 2^-24, one FP32 rounding): a row's sum of squares is right to 100 u (64 + 16 steps a thread and a tree of
positive terms), its root to 60 u with the square root, the divisions and eps.  gate u carries that and four products;
h one more rounding.  The second norm's factor adds what h's errors are of its norm.  y is three products and a sum.  A
rotated element adds log2 b sums none larger than its block's L1 norm.  Codes and bf16 are half a step on top.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _half_ulp(v):
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -126))) - 8)


def _sylvester(b):
    h = np.ones((1, 1))
    while h.shape[0] < b:
        h = np.block([[h, h], [h, -h]])
    return h


def _inputs(m, k, seed, residual=True, weight=True, post=True, mod="all", segments=1, indexed=False):
    g = np.random.default_rng(seed)

    def bf16(a):
        return torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).float().numpy()

    x = g.laplace(size=(m, k))
    x[:, g.random(k) < 0.005] *= 50
    c = dict(x=bf16(x), res=bf16(g.normal(size=(m, k))) if residual else None)
    c["w"] = (g.random(k) + 0.5).astype(np.float32) if weight else None
    c["post"] = (g.random(k) + 0.5).astype(np.float32) if post else None
    for name, on in (("gate", mod != "none"), ("scale", mod == "all"), ("shift", mod == "all")):
        c[name] = (g.normal(size=(segments, k)) * 0.5).astype(np.float32) if on else None
    c["segment"] = g.integers(0, segments, m).astype(np.int32) if indexed else None
    c["S"], c["rs"] = segments, 0.75
    return c


def _ref(c, b):
    """(h, its error, z, its error) in float64."""
    x = c["x"].astype(np.float64)
    m, k = x.shape
    at = c["segment"] if c["segment"] is not None else np.arange(m) // max(1, m // c["S"])
    f = {n: None if c[n] is None else c[n].astype(np.float64)[at] for n in ("gate", "scale", "shift")}
    u = x
    if c["post"] is not None:
        u = x / np.sqrt((x * x).mean(1, keepdims=True) + EPS) * c["post"]
    if f["gate"] is not None:
        u = u * f["gate"]
    h = u + (0 if c["res"] is None else c["rs"] * c["res"].astype(np.float64))
    eh = 64 * U * np.abs(u) + U * np.abs(h)
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + EPS)
    w = np.ones(k) if c["w"] is None else c["w"].astype(np.float64)
    if f["scale"] is not None:
        w = w * (1 + f["scale"])
    y = h * r * w
    rho = np.linalg.norm(eh, axis=1, keepdims=True) / np.maximum(np.linalg.norm(h, axis=1, keepdims=True), 1e-300) + 60 * U
    ey = r * np.abs(w) * eh + np.abs(y) * (rho + 4 * U)
    if f["shift"] is not None:
        y = y + f["shift"]
        ey = ey + U * np.abs(y)
    if b:
        z = (y.reshape(m, k // b, b) @ _sylvester(b)).reshape(m, k) / np.sqrt(b)

        def l1(v):
            return np.repeat(v.reshape(m, k // b, b).sum(2), b, 1) / np.sqrt(b)

        ez = l1(ey) + np.log2(b) * U * l1(np.abs(y))
    else:
        z, ez = y, ey
    return h, eh, z, ez


def _call(ops, c, b, **kw):
    def dev(a, dtype=torch.float32):
        return None if a is None else torch.from_numpy(a).to(dtype).cuda()

    mods = {n: dev(c[n]) for n in ("gate", "scale", "shift")}
    x, res = dev(c["x"], torch.bfloat16), dev(c["res"], torch.bfloat16)
    return ops.gated_rmsnorm_quant(x, res, dev(c["w"]), post_weight=dev(c["post"]), segment=dev(c["segment"], torch.int32),
                                   residual_scale=c["rs"], eps=EPS, had_block=b, **mods, **kw)


def _check_sum(h, want, err):
    got = h.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= err + _half_ulp(np.abs(want) + err)), "sum"


def _check(ops, c, b, rows=slice(None), got=None):
    a, h = _call(ops, c, b) if got is None else got
    want, eh, z, ez = _ref(c, b)
    _check_sum(h[rows], want[rows], eh[rows])
    q = a.i8_codes.cpu().numpy().astype(np.float64)[rows]
    s = a.row_scale.cpu().numpy().astype(np.float64)[rows]
    z, ez = z[rows], ez[rows]
    top = np.abs(z).max(1)
    assert np.all(np.abs(s * 127 - top) <= ez.max(1) + 4 * U * top), "row scale"
    assert np.all(np.abs(q * s[:, None] - z) <= s[:, None] * (0.5 + 127 * 8 * U) + 2 * ez.max(1, keepdims=True)), "codes"
    assert np.all(np.abs(q).max(1)[top > 0] == 127)


@pytest.mark.parametrize("b", [0, 16, 64, 256])
@pytest.mark.parametrize("m,k", [(1, 256), (3, 512), (37, 768), (200, 1280), (5, 4096), (17, 4352), (9, 8448), (3, 16384)])
def test_shapes(ops, m, k, b):
    _check(ops, _inputs(m, k, 100 * b + k + m), b)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("mod", ["none", "gate", "all"])
@pytest.mark.parametrize("m,k,b", [(1, 128, 64), (33, 1920, 64), (7, 12288, 0)])
def test_optional_operands(ops, m, k, b, residual, weight, post, mod):
    _check(ops, _inputs(m, k, m + k, residual, weight, post, mod), b)


@pytest.mark.parametrize("m,segments,indexed", [(700, 7, False), (701, 7, True), (4000, 2, False), (1501, 40, True)])
def test_segments(ops, m, segments, indexed):
    for mod in ("gate", "all"):
        _check(ops, _inputs(m, 384, m, mod=mod, segments=segments, indexed=indexed), 64)


@pytest.mark.parametrize("k", [128, 640, 1024, 1920, 2048, 2176, 4096, 5120, 7680, 8192, 8320, 16384])
@pytest.mark.parametrize("m,b", [(600, 64), (1217, 0), (2500, 16)])
def test_many_rows(ops, m, k, b):
    """Rows whose parts are copied ahead, teams of every size, windows of segments that do not all fit."""
    for segments, indexed in ((1, False), (11, True)):
        _check(ops, _inputs(m, k, m + k, segments=segments, indexed=indexed), b)
    c = _inputs(m, k, k, segments=5)
    c["segment"] = np.sort(np.random.default_rng(m).integers(0, 5, m)).astype(np.int32)  # runs
    _check(ops, c, b)
    c["res"] = None
    c["post"] = None
    _check(ops, c, b)


@pytest.mark.parametrize("k", [256, 1920, 7680, 16384])
def test_many_rows_in_place_and_bf16(ops, k):
    m = 777
    c = _inputs(m, k, k, segments=3)
    want, hw = _call(ops, c, 64)
    f = {n: torch.from_numpy(c[n]).cuda() for n in ("w", "post", "gate", "scale", "shift")}
    for i in range(2):
        v = [torch.from_numpy(c[n]).to(torch.bfloat16).cuda() for n in ("x", "res")]
        a, h = ops.gated_rmsnorm_quant(*v, f["w"], f["post"], f["gate"], f["scale"], f["shift"], None, 0.75, EPS, 64,
                                       sum_out=v[i])
        assert h is v[i] and torch.equal(h, hw)
        assert torch.equal(a.i8_codes, want.i8_codes) and torch.equal(a.row_scale, want.row_scale)
    y, h = _call(ops, c, 0, quantize=False)
    _, _, z, ez = _ref(c, 0)
    assert torch.equal(h, hw)
    assert np.all(np.abs(y.double().cpu().numpy() - z) <= ez + _half_ulp(np.abs(z) + ez))


def test_many_special_rows(ops):
    m, k = 700, 1920
    c = _inputs(m, k, 2, segments=2, indexed=True)
    bad = [3, 77, 333, 699]
    c["x"][3, 5], c["res"][77, 9], c["x"][333, 0] = np.inf, np.nan, -np.inf
    c["segment"][699] = 2
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, h = _call(ops, c, 64, err=err)
    with pytest.raises(RuntimeError):
        ops.check_err(err, "norm")
    s = a.row_scale.cpu().numpy()
    assert np.isnan(s[bad]).all() and not a.i8_codes[bad].any()
    for i in bad:
        c["x"][i], c["res"][i], c["segment"][i] = 1, 1, 0
    _check(ops, c, 64, rows=[i for i in range(m) if i not in bad], got=(a, h))


@pytest.mark.parametrize("one", ["gate", "scale", "shift"])
def test_one_modulation_alone(ops, one):
    c = _inputs(41, 640, 3, segments=3, indexed=True)
    for n in ("gate", "scale", "shift"):
        if n != one:
            c[n] = None
    _check(ops, c, 64)
    c = _inputs(900, 1280, 3, residual=False, post=False, weight=False, segments=3, indexed=True)
    for n in ("gate", "scale", "shift"):
        if n != one:
            c[n] = None
    _check(ops, c, 64)


@pytest.mark.parametrize("m,k", [(1, 128), (50, 1920), (1003, 640), (5, 8448)])
@pytest.mark.parametrize("post", [False, True])
def test_bf16_result(ops, m, k, post):
    c = _inputs(m, k, m, post=post, segments=3, indexed=True)
    y, h = _call(ops, c, 0, quantize=False)
    want, eh, z, ez = _ref(c, 0)
    _check_sum(h, want, eh)
    assert y.dtype == torch.bfloat16
    assert np.all(np.abs(y.double().cpu().numpy() - z) <= ez + _half_ulp(np.abs(z) + ez))


@pytest.mark.parametrize("k", [256, 1920, 12288])
def test_special_rows(ops, k):
    c = _inputs(10, k, k, segments=2, indexed=True)
    x, r = c["x"], c["res"]
    x[1], r[1] = 0, 0                 # the shift alone
    x[2], r[2] = 0, 0
    x[2, k - 1] = 3.0
    x[4, 5] = np.inf
    r[5, k - 3] = np.nan
    x[6, 0], r[6, 0] = np.inf, -np.inf
    x[7, :] = 3e38                    # the branch's sum of squares overflows
    r[8, :] = 3e38                    # the stream's does
    got = _call(ops, c, 64)
    s, q = got[0].row_scale.cpu().numpy(), got[0].i8_codes.cpu().numpy()
    bad = [4, 5, 6, 7, 8]
    assert np.isnan(s[bad]).all() and not q[bad].any()
    fine = [i for i in range(10) if i not in bad]
    for i in bad:
        x[i], r[i] = 1, 1             # (the reference of the others alone)
    _check(ops, c, 64, rows=fine, got=got)
    for n in ("scale", "shift", "gate"):
        c[n] = None
    x[1], r[1] = 0, 0
    a, _ = _call(ops, c, 64)
    assert float(a.row_scale[1]) == 0 and not a.i8_codes[1].any()


def test_the_smallest_values(ops):
    c = _inputs(4, 256, 1, post=False, mod="none", weight=False)
    c["res"][:] = 0
    c["x"][1:] = torch.from_numpy(c["x"][1:] * 1e-36).to(torch.bfloat16).float().numpy()
    _check(ops, c, 64)


def test_a_segment_out_of_range_is_reported(ops):
    c = _inputs(9, 384, 5, segments=3, indexed=True)
    c["segment"][[2, 7]] = [-1, 3]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, h = _call(ops, c, 64, err=err)
    with pytest.raises(RuntimeError):
        ops.check_err(err, "norm")
    s = a.row_scale.cpu().numpy()
    assert np.isnan(s[[2, 7]]).all() and not a.i8_codes[[2, 7]].any() and torch.isnan(h[[2, 7]].float()).all()
    c["segment"][[2, 7]] = 0
    _check(ops, c, 64, rows=[0, 1, 3, 4, 5, 6, 8], got=(a, h))
    y, _ = _call(ops, dict(c, segment=np.full(9, 9, np.int32)), 0, quantize=False)
    assert torch.isnan(y.float()).all()


def test_with_nothing_but_a_residual_it_is_add_rmsnorm_quant(ops):
    """The same norm with the branch ungated: codes and sums of the two calls agree but for ties."""
    c = _inputs(64, 1920, 9, post=False, mod="none")
    c["rs"] = 1.0
    x, r, w = (torch.from_numpy(c[n]).cuda() for n in ("x", "res", "w"))
    x, r = x.to(torch.bfloat16), r.to(torch.bfloat16)
    a, h = ops.add_rmsnorm_quant(x, r, w, had_block=64)
    b, h2 = ops.gated_rmsnorm_quant(x, r, w, had_block=64)
    assert torch.equal(h, h2)
    assert int((a.i8_codes.int() - b.i8_codes.int()).abs().max()) <= 1
    assert torch.allclose(a.row_scale, b.row_scale, rtol=1e-6, atol=0)


@pytest.mark.parametrize("k", [256, 1920, 8448])
def test_in_place_alignment_stream_and_mode(ops, k):
    c = _inputs(19, k, 3 * k, segments=2, indexed=True)
    want, hw = _call(ops, c, 64)

    def same(a, h):
        assert torch.equal(h, hw) and torch.equal(a.i8_codes, want.i8_codes) and torch.equal(a.row_scale, want.row_scale)

    f = {n: torch.from_numpy(c[n]).cuda() for n in ("w", "post", "gate", "scale", "shift", "segment")}

    def call(x, r, **kw):
        return ops.gated_rmsnorm_quant(x, r, f["w"], f["post"], f["gate"], f["scale"], f["shift"], f["segment"], 0.75,
                                       EPS, 64, **kw)

    def fresh():
        return tuple(torch.from_numpy(c[n]).to(torch.bfloat16).cuda() for n in ("x", "res"))

    for i in range(2):
        v = fresh()
        a, h = call(*v, sum_out=v[i])
        assert h is v[i]
        same(a, h)

    def at16(v):  # 16-byte but not 32-byte aligned
        buf = torch.empty(v.numel() + 8, dtype=v.dtype, device="cuda")
        o = buf[8:].view(v.shape)
        o.copy_(v)
        assert o.data_ptr() % 32 == 16
        return o

    same(*call(*(at16(v) for v in fresh())))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    v = fresh()
    torch.cuda.synchronize()
    got = call(*v, stream=side)
    side.synchronize()
    same(*got)
    mode = torch.tensor([ops.MODE_BF16], dtype=torch.int32, device="cuda")
    a, h = ops.int8_act(torch.full((19, k), 3, dtype=torch.int8, device="cuda"), torch.full((19,), 2.0, device="cuda")), v[0]
    before = h.clone()
    call(*v, out=a, sum_out=h, mode_dev=mode)
    assert torch.equal(h, before) and bool((a.i8_codes == 3).all()) and bool((a.row_scale == 2).all())
    mode.fill_(ops.MODE_INT8)
    same(*call(*v, out=a, sum_out=h, mode_dev=mode))


def test_captured(ops):
    c = _inputs(33, 640, 1, segments=2, indexed=True)
    want, hw = _call(ops, c, 64)
    f = {n: torch.from_numpy(c[n]).cuda() for n in ("w", "post", "gate", "scale", "shift", "segment")}
    x, r = (torch.from_numpy(c[n]).to(torch.bfloat16).cuda() for n in ("x", "res"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, h = ops.gated_rmsnorm_quant(x, r, f["w"], f["post"], f["gate"], f["scale"], f["shift"], f["segment"], 0.75,
                                       EPS, 64)
    for _ in range(2):
        a.i8_codes.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.i8_codes, want.i8_codes) and torch.equal(h, hw) and torch.equal(a.row_scale, want.row_scale)


def test_beyond_32_bit_offsets(ops):
    m, k = 1_130_000, 1920  # 2.17e9 elements
    c = _inputs(3, k, 5)
    x = torch.zeros((m, k), dtype=torch.bfloat16, device="cuda")
    r = torch.zeros_like(x)
    rows = torch.tensor([0, m // 2 + 1, m - 1]).cuda()
    x[rows] = torch.from_numpy(c["x"]).to(torch.bfloat16).cuda()
    r[rows] = torch.from_numpy(c["res"]).to(torch.bfloat16).cuda()
    f = {n: torch.from_numpy(c[n]).cuda() for n in ("w", "post", "gate", "scale", "shift")}
    a, h = ops.gated_rmsnorm_quant(x, r, f["w"], f["post"], f["gate"], f["scale"], f["shift"], None, 0.75, EPS, 64,
                                   sum_out=r)
    _check(ops, c, 64, got=(ops.int8_act(a.i8_codes[rows], a.row_scale[rows]), h[rows]))
    assert int((h != 0).any(1).sum()) == 3


def test_empty_and_refusals(ops):
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    g = torch.zeros((2, 256), device="cuda")
    a, h = ops.gated_rmsnorm_quant(x[:0], gate=g)
    assert a.m == 0 and h.shape == (0, 256)
    y, _ = ops.gated_rmsnorm_quant(x[:0], quantize=False)
    assert y.shape == (0, 256)
    f = torch.zeros(256, device="cuda")
    for bad in (lambda: ops.gated_rmsnorm_quant(x.float()), lambda: ops.gated_rmsnorm_quant(x[0]),
                lambda: ops.gated_rmsnorm_quant(x.cpu()), lambda: ops.gated_rmsnorm_quant(x, x[:2]),
                lambda: ops.gated_rmsnorm_quant(x, weight=f[:128]), lambda: ops.gated_rmsnorm_quant(x, gate=g.half()),
                lambda: ops.gated_rmsnorm_quant(x, gate=g, shift=f), lambda: ops.gated_rmsnorm_quant(x, gate=g, scale=g[:1]),
                lambda: ops.gated_rmsnorm_quant(x, gate=f, scale=g), lambda: ops.gated_rmsnorm_quant(x[:3], gate=g),
                lambda: ops.gated_rmsnorm_quant(x, gate=g, segment=torch.zeros(4, device="cuda")),
                lambda: ops.gated_rmsnorm_quant(x, gate=g, segment=torch.zeros(3, dtype=torch.int32, device="cuda")),
                lambda: ops.gated_rmsnorm_quant(x[:, ::2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.gated_rmsnorm_quant(x, had_block=64, quantize=False), lambda: ops.gated_rmsnorm_quant(x, eps=0.0),
                lambda: ops.gated_rmsnorm_quant(x, residual_scale=float("inf")), lambda: ops.gated_rmsnorm_quant(x, had_block=32)):
        with pytest.raises(RuntimeError):
            bad()
