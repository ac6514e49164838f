"""Routing against its definition in 64 bits: experts, rows and offsets equal, weights to FP32.

Weights: an exponential is right to 2 u' (u' = 2^-23) and its argument l - m to 2^-24 |l - m|; a sum of E of them to
(E / 32 + 5) 2^-24 more; then a division and two products.  With logits below 30 in size: 2^-24 (4 + 60 + E / 32 + 13) of
the weight, twice for numerator and sum.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _ref(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, best=2, renorm=True, scale=1.0):
    """float64, one token after the other."""
    z = logits.double().numpy()
    t, e = z.shape
    with np.errstate(over="ignore"):
        p = 1 / (1 + np.exp(-z)) if sigmoid else np.exp(z - z.max(1, keepdims=True))
    if not sigmoid:
        p = p / p.sum(1, keepdims=True)
    key = p if bias is None else p + bias.double().numpy()
    experts, weights = np.zeros((t, k), np.int64), np.zeros((t, k))
    size = e // groups
    for i in range(t):
        allowed = np.arange(e)
        if groups > 1:
            g = np.sort(key[i].reshape(groups, size), 1)[:, ::-1][:, :best].sum(1)
            kept = np.argsort(-g, kind="stable")[:top_groups]
            allowed = np.array([x for x in range(e) if x // size in kept])
        order = (z if bias is None else key)[i][allowed]
        chosen = allowed[np.argsort(-order, kind="stable")[:k]]
        experts[i] = chosen
        w = p[i][chosen]
        if renorm:
            if sigmoid:  # (the ratio of the smallest scores)
                w = np.where(z[i][chosen] == -np.inf, 0, w)
            else:
                m = z[i][chosen].max()
                w = np.exp(z[i][chosen] - m) if m > -np.inf else np.zeros(k)
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        weights[i] = w * scale
    return experts, weights


def _check(r, experts, weights, e):
    t, k = experts.shape
    assert np.array_equal(r.experts.cpu().numpy(), experts), "experts"
    tol = 2.0 ** -24 * 2 * (77 + e / 32) * np.abs(weights) + 1e-37
    assert np.all(np.abs(r.weights.double().cpu().numpy() - weights) <= tol), "weights"
    _check_places(r, e)


def _check_places(r, e):
    ex = r.experts.cpu().numpy()
    t, k = ex.shape
    order = np.argsort(ex.reshape(-1), kind="stable")
    rows = np.empty(t * k, np.int64)
    rows[order] = np.arange(t * k)
    assert np.array_equal(r.rows.cpu().numpy().reshape(-1), rows), "rows"
    assert np.array_equal(r.token.cpu().numpy(), order // k), "tokens"
    counts = np.bincount(ex.reshape(-1), minlength=e)
    assert np.array_equal(r.offsets.cpu().numpy(), np.concatenate(([0], np.cumsum(counts)))), "offsets"
    for v in (r.experts, r.rows, r.token, r.offsets):
        assert v.dtype == torch.int32 and v.is_contiguous()


def _logits(t, e, seed, dtype=torch.float32, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((t, e), generator=g) * spread).to(dtype), torch.randn(e, generator=g) * 0.2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("t,e,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (31, 33, 8), (32, 64, 2), (33, 64, 6), (200, 100, 3),
                                   (700, 256, 8), (40, 600, 32), (257, 1024, 9), (3000, 16, 1)])
def test_choice(ops, t, e, k, sigmoid, dtype):
    z, bias = _logits(t, e, t + e + k, dtype)
    score = ops.SCORE_SIGMOID if sigmoid else ops.SCORE_SOFTMAX
    for b in (None, bias):
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            r = ops.moe_route(z.cuda(), k, score, bias=None if b is None else b.cuda(), renormalize=renorm, scale=scale)
            _check(r, *_ref(z, k, sigmoid, b, renorm=renorm, scale=scale), e)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("t,e,groups,top,best,k", [(1, 8, 4, 2, 2, 3), (50, 256, 8, 4, 2, 8), (300, 96, 32, 5, 1, 6),
                                                   (65, 60, 6, 1, 2, 10), (40, 21, 7, 3, 2, 4), (33, 32, 32, 4, 2, 4),
                                                   (70, 1024, 16, 3, 2, 12), (100, 48, 3, 3, 1, 5)])
def test_groups(ops, t, e, groups, top, best, k, sigmoid):
    z, bias = _logits(t, e, t + e + groups)
    score = ops.SCORE_SIGMOID if sigmoid else ops.SCORE_SOFTMAX
    for b in (None, bias):
        r = ops.moe_route(z.cuda(), k, score, bias=None if b is None else b.cuda(), groups=groups, top_groups=top,
                          group_best=best)
        _check(r, *_ref(z, k, sigmoid, b, groups, top, best), e)


@pytest.mark.parametrize("e,k,groups", [(8, 2, 1), (64, 4, 1), (64, 4, 8), (300, 8, 1), (256, 8, 8)])
def test_keys_that_fp32_cannot_tell_apart(ops, e, k, groups):
    """The bias cancels the score: all keys lie within a few 2^-24, and FP64 decides."""
    t = 150
    z, _ = _logits(1, e, e, spread=1.0)
    bias = (0.75 - torch.sigmoid(z.double())).float()[0]
    z = z.expand(t, e).clone()
    g = torch.Generator().manual_seed(1)
    z += torch.randn((t, e), generator=g) * 1e-7  # (a few units of a logit)
    kw = dict(groups=groups, top_groups=max(1, groups // 2), best=2)
    want = _ref(z, k, True, bias, **kw)
    r = ops.moe_route(z.cuda(), k, ops.SCORE_SIGMOID, bias=bias.cuda(), groups=groups, top_groups=kw["top_groups"])
    _check(r, *want, e)


def test_ties_go_to_the_lower_number(ops):
    z = torch.zeros((70, 48))
    z[:, 40] = 1.0
    z[1::2, 7] = 1.0
    z[0, 3] = -0.0
    for sigmoid in (False, True):
        for b in (None, torch.zeros(48)):
            for groups in (1, 4):
                r = ops.moe_route(z.cuda(), 4, int(sigmoid), bias=None if b is None else b.cuda(), groups=groups,
                                  top_groups=min(2, groups))
                _check(r, *_ref(z, 4, sigmoid, b, groups, min(2, groups)), 48)
    big = torch.full((5, 20), 50.0)  # sigmoid is 1 in 64 bits too
    r = ops.moe_route(big.cuda(), 3, ops.SCORE_SIGMOID, bias=torch.zeros(20).cuda())
    assert r.experts.tolist() == [[0, 1, 2]] * 5


def test_infinite_logits(ops):
    z, _ = _logits(40, 12, 3)
    z[:, 5] = -np.inf
    z[1, :] = -np.inf
    z[2, 1:] = -np.inf
    for sigmoid in (False, True):
        keep = [i for i in range(40) if sigmoid or i != 1]
        r = ops.moe_route(z.cuda(), 3, int(sigmoid))
        ex, w = _ref(z[keep], 3, sigmoid)
        assert np.array_equal(r.experts.cpu().numpy()[keep], ex)
        assert np.allclose(r.weights.cpu().numpy()[keep], w, rtol=1e-5, atol=0)
        assert r.experts[1].tolist() == [0, 1, 2] and not r.weights[1].any()  # nothing is left: weights of 0
        assert r.weights[2].tolist() == [1.0, 0.0, 0.0]
        _check_places(r, 12)
        r = ops.moe_route(z.cuda(), 3, int(sigmoid), renormalize=False)
        assert not r.weights[1].any() and torch.isfinite(r.weights).all()
    z[3, 4] = np.inf
    r = ops.moe_route(z.cuda(), 2)
    assert r.experts[3, 0] == 4 and torch.isnan(r.weights[3]).all() and not torch.isnan(r.weights[4:]).any()
    r = ops.moe_route(z.cuda(), 2, ops.SCORE_SIGMOID, renormalize=False)
    assert r.experts[3, 0] == 4 and r.weights[3, 0] == 1


@pytest.mark.parametrize("e,k,groups", [(12, 2, 1), (12, 6, 3), (64, 8, 1), (64, 5, 8), (300, 10, 1), (300, 12, 4)])
def test_infinite_and_nan_biases(ops, e, k, groups):
    """Biases that put experts in front of or behind all others."""
    z, bias = _logits(37, e, e + k)
    for n, value in ((1, np.inf), (k - 1, np.inf), (k + 3, np.inf), (1, -np.inf), (e // 2, -np.inf), (e - 1, -np.inf), (2, 3e38)):
        b = bias.clone()
        b[torch.randperm(e, generator=torch.Generator().manual_seed(n))[:n]] = value
        for score in (0, 1):
            kw = dict(groups=groups, top_groups=(groups + 1) // 2)
            if groups > 1 and value < 0:
                continue  # (whole groups of the same score: any of them)
            r = ops.moe_route(z.cuda(), k, score, bias=b.cuda(), **kw)
            ex, w = _ref(z, k, bool(score), b, **kw)
            assert np.array_equal(r.experts.cpu().numpy(), ex)
            assert np.allclose(r.weights.cpu().numpy(), w, rtol=1e-5, atol=1e-30)
            _check_places(r, e)
    bias[[3, 5]] = np.nan  # first, by their numbers
    r = ops.moe_route(z.cuda(), k, 1, bias=bias.cuda())
    assert bool((r.experts[:, :2].cpu() == torch.tensor([3, 5])).all())
    _check_places(r, e)
    for value in (np.nan, np.inf, -np.inf):
        r = ops.moe_route(z.cuda(), k, 1, bias=torch.full((e,), float(value)).cuda(), groups=groups, top_groups=groups)
        assert bool((r.experts.cpu() == torch.arange(k)).all())  # all alike
        _check_places(r, e)


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("with_bias", [False, True])
def test_nan_logits_stay_in_their_row(ops, with_bias, groups):
    z, bias = _logits(50, 12, 4)
    fine = z.clone()
    z[7, 9] = np.nan
    b = bias.cuda() if with_bias else None
    for score in (0, 1):
        kw = dict(bias=b, groups=groups, top_groups=min(2, groups))
        r, f = ops.moe_route(z.cuda(), 2, score, **kw), ops.moe_route(fine.cuda(), 2, score, **kw)
        assert torch.isnan(r.weights[7]).all()
        assert score == 0 and (with_bias or groups > 1) or r.experts[7, 0] == 9
        rest = [i for i in range(50) if i != 7]
        assert torch.equal(r.experts[rest], f.experts[rest]) and torch.equal(r.weights[rest], f.weights[rest])
        assert bool(((r.experts >= 0) & (r.experts < 12)).all()) and r.experts[7, 0] != r.experts[7, 1]
        _check_places(r, 12)


def test_small_scores_keep_their_ratio(ops):
    """Chosen by the bias although their scores underflow FP32: the renormalised weights are still their ratio."""
    z = torch.full((2, 8), -120.0)
    z[:, 0], z[:, 3] = 10.0, -121.0
    bias = torch.zeros(8)
    bias[2], bias[3] = 5.0, 4.0
    for score in (0, 1):
        r = ops.moe_route(z.cuda(), 2, score, bias=bias.cuda())
        e = 1 / (1 + np.exp(-1.0))
        assert r.experts.tolist() == [[2, 3]] * 2
        assert np.allclose(r.weights.cpu().numpy(), [[e, 1 - e]] * 2, rtol=1e-5)


@pytest.mark.parametrize("t", [20_000, 100_003])
def test_long(ops, t):
    z, _ = _logits(t, 32, t)
    r = ops.moe_route(z.cuda(), 2)
    assert torch.equal(r.experts.cpu().long(), z.sort(dim=1, descending=True, stable=True).indices[:, :2])
    _check_places(r, 32)


def test_repeats_streams_and_graphs(ops):
    z, bias = _logits(900, 64, 8)
    zd, bd = z.cuda(), bias.cuda()

    def call(**kw):
        return ops.moe_route(zd, 4, ops.SCORE_SIGMOID, bias=bd, groups=8, top_groups=3, **kw)

    want = call()
    _check(want, *_ref(z, 4, True, bias, 8, 3), 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = [call() for _ in range(20)] + [call(stream=side) for _ in range(20)]
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call()
    for _ in range(3):
        for v in r:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_empty_and_refusals(ops):
    z = torch.zeros((4, 12), device="cuda")
    r = ops.moe_route(z[:0], 2)
    assert r.experts.shape == r.weights.shape == r.rows.shape == (0, 2) and r.offsets.tolist() == [0] * 13
    for bad in (lambda: ops.moe_route(z.cpu(), 2), lambda: ops.moe_route(z.half(), 2), lambda: ops.moe_route(z[0], 2),
                lambda: ops.moe_route(z, 13), lambda: ops.moe_route(z, 0), lambda: ops.moe_route(z[:, ::2], 2),
                lambda: ops.moe_route(z, 2, bias=z[0, :5]), lambda: ops.moe_route(z, 2, bias=torch.zeros(12))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.moe_route(z, 2, 2), lambda: ops.moe_route(z, 2, groups=5), lambda: ops.moe_route(z, 5, groups=3, top_groups=1),
                lambda: ops.moe_route(z, 2, groups=3, top_groups=4), lambda: ops.moe_route(z, 2, groups=0),
                lambda: ops.moe_route(z, 2, group_best=3), lambda: ops.moe_route(z, 2, scale=float("nan")),
                lambda: ops.moe_route(torch.zeros((2, 1025), device="cuda"), 1)):
        with pytest.raises(RuntimeError):
            bad()
