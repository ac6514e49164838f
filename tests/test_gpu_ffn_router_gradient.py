"""MoEFFN's router can be trained: its gradient through y and through route()'s weights is that of topk, softmax and a
weighted sum, and agrees with differences."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ffn():
    from video_dit_mixed_gb300 import ffn as f
    return f


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _layer(ffn, ops, t, e=8, k=2, hid=128, f=256, b=16, seed=0, trained=True, **kw):
    g = torch.Generator().manual_seed(seed + t)
    up, down = (ops.pack_experts((torch.randn((e,) + s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))
    router = (torch.randn((e, hid), generator=g) * 0.3).cuda().requires_grad_(trained)
    x, r = (torch.randn((t, hid), generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    return ffn.MoEFFN(router, up, down, k, had_block=b, **kw), router, x, r, g


@pytest.mark.parametrize("normed", [False, True])
@pytest.mark.parametrize("t,e,k", [(1, 8, 2), (70, 8, 1), (70, 8, 3), (40, 40, 36)])
def test_default_rule(ffn, ops, t, e, k, normed):
    layer, router, x, r, g = _layer(ffn, ops, t, e, k, normed_router=normed)
    y, h = layer(x, r)
    assert y.requires_grad
    dy = torch.randn(y.shape, generator=g).to(torch.bfloat16).cuda()
    got, = torch.autograd.grad(y, router, dy)

    logits = h.float() @ router.mT
    if normed:
        logits = logits * torch.rsqrt(h.float().square().mean(1, keepdim=True) + layer.eps)
    top = logits.topk(k, dim=1)
    weights = torch.softmax(top.values, dim=1)
    rows, w, token, offsets = layer.route(h)
    assert w.requires_grad and torch.equal(w, weights)
    a, _ = ops.add_rmsnorm_quant(x, r, None, layer.eps, layer.had_block)
    u = ops.qgemm_grouped(ops.int8_act(a.i8_codes[token], a.row_scale[token]), layer.up, offsets, ops.EPI_GELU)
    q = ops.hadamard_quant(u, layer.had_block, ops.MODE_INT8, out=ops.QActTensors(*u.shape, u.device, nvfp4=False))
    d = ops.qgemm_grouped(q, layer.down, offsets, out_f32=True)
    ref = (d[rows] * weights.unsqueeze(-1)).sum(1).to(torch.bfloat16)
    assert torch.equal(y, ref)
    want, = torch.autograd.grad(ref, router, dy)
    assert torch.equal(got, want) or float((got - want).norm()) <= 2.0 ** -18 * float(want.norm())  # (atomics of the gathers)
    dw = torch.randn(w.shape, generator=g).cuda()
    got, = torch.autograd.grad(w, router, dw)
    logits = h.float() @ router.mT
    if normed:
        logits = logits * torch.rsqrt(h.float().square().mean(1, keepdim=True) + layer.eps)
    want, = torch.autograd.grad(torch.softmax(logits.topk(k, dim=1).values, 1), router, dw)
    assert float((got - want).norm()) <= 2.0 ** -18 * float(want.norm()) + 1e-12


@pytest.mark.parametrize("rule", [dict(score=1, route_scale=2.5), dict(score=1, bias=True, groups=4, top_groups=2),
                                  dict(bias=True, renormalize=False), dict(score=1, renormalize=False),
                                  dict(groups=2, top_groups=1, group_best=1)])
def test_other_rules(ffn, ops, rule):
    """Against float64 and its differences, with the experts that were chosen.  The weights agree to FP32's errors (an
    exponential of a logit below 16 in size, a sum and a division: 2^-19); the gradient is a sum over 60 tokens of products
    of them: 2^-15 of its norm.  A central difference with a step of 2^-10 is off by a sixth of 2^-20 of a third derivative."""
    rule = dict(rule)
    g = torch.Generator().manual_seed(4)
    bias = (torch.randn(8, generator=g) * 0.2).cuda() if rule.pop("bias", False) else None
    t, e, k = 60, 8, 2
    layer, router, x, r, g = _layer(ffn, ops, t, e, k, bias=bias, **rule)
    _, h = layer(x, r)
    rows, w, token, offsets = layer.route(h)
    experts = torch.searchsorted(offsets[1:].long(), rows, right=True)
    plain = ops.moe_route(layer.logits(h).detach(), k, **layer.rule)
    assert torch.equal(plain.experts.long(), experts) and torch.equal(plain.rows.long(), rows)
    v = w.detach()
    assert float((v - plain.weights).abs().max()) <= 2.0 ** -19 * float(v.abs().max())
    dw = torch.randn(w.shape, generator=g).double()

    def weights(m):
        z = h.double().cpu() @ m.mT
        p = torch.sigmoid(z) if rule.get("score") else torch.softmax(z, 1)
        v = p.gather(1, experts.cpu())
        if rule.get("renormalize", True):
            v = v / v.sum(1, keepdim=True)
        return v * rule.get("route_scale", 1.0)

    m = router.detach().double().cpu().requires_grad_()
    want, = torch.autograd.grad(weights(m), m, dw)
    got = torch.autograd.grad(w, router, dw.float().cuda())[0].double().cpu()
    assert float((got - want).norm()) <= 2.0 ** -15 * float(want.norm())
    with torch.no_grad():
        way = torch.randn(m.shape, generator=g).double()
        way /= (h.double().cpu() @ way.mT).abs().max()
        s = 2.0 ** -10
        diff = ((weights(m + s * way) - weights(m - s * way)) * dw).sum() / (2 * s)
        assert abs(float(diff - (got * way).sum())) <= 1e-4 * float((weights(m) * dw).abs().sum())


def test_values_do_not_depend_on_training(ffn, ops):
    for t in (1, 90):
        layer, router, x, r, _ = _layer(ffn, ops, t)
        y, h = layer(x, r)
        with torch.no_grad():
            y2, h2 = layer(x, r)
        assert y.requires_grad and not y2.requires_grad and torch.equal(y, y2) and torch.equal(h, h2)
