"""The feed-forward layers with a block's gate, norms and modulation, with adapters, and with every rule of routing,
against the same layer in 64 bits on the packed weights.

The reference quantizes its own activations in float64 and rounds u to bf16, so y agrees in norm: u's roundings are 2^-9
each, a flipped code moves one term of a sum of hundreds by 1/127 of its row's largest, the adapters' A is rounded to bf16
behind its rotation (2^-9), and the output's own rounding is 2^-9.  Bound: 2^-7.

With adapters 2^-6.  The reference's A is not rounded, so its u differs: A's roundings are 0.0017 of A in norm (a
uniform error of half a step, 2^-9 to 2^-8 of a value), 0.0012 of u where the adapter makes 0.7 of it; two roundings to
steps of 2^-8 of values 0.0012 apart differ by sqrt(0.0012 x 2^-8) = 0.002 in the mean square; together d = 0.0024 of u.
Quantizing u turns a difference of |d| on average 0.8 d into one of sqrt(0.8 d s) in the mean square, s = the step, a
127th of a row's largest: with 640 values 3.2 / 127 = 0.025 of their size.  That is 0.0069, and with A's and the
output's roundings behind it 0.0073 on average; 2^-6 = 0.0156 leaves a factor of two for the smallest batches.
"""
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


def _rotate(y, b):
    h = torch.ones((1, 1), dtype=torch.float64)
    while h.shape[0] < b:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)))
    return (y.reshape(-1, b) @ h / b ** 0.5).reshape(y.shape)


def _quantized(y):
    s = y.abs().amax(1, keepdim=True) / 127
    return torch.round(y / s.clamp(min=1e-300)) * s


def _weight(codes, scales):
    c = codes.cpu().to(torch.int16)
    q = (torch.stack((c & 15, c >> 4), -1).flatten(1) ^ 8) - 8
    return q.double() * scales.cpu().double().repeat_interleave(128, 0).mT


def _rms(v):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6)


def _stream(c):
    """(h, the norm's output) in float64."""
    u = c["x"].double()
    if c["post"] is not None:
        u = _rms(u) * c["post"].double()
    if c["gate"] is not None:
        u = u * c["gate"].double()[c["seg"]]
    h = u + c["rs"] * c["r"].double()
    y = _rms(h) * c["nw"].double()
    if c["scale"] is not None:
        y = y * (1 + c["scale"].double()[c["seg"]])
    if c["shift"] is not None:
        y = y + c["shift"].double()[c["seg"]]
    return h, y


def _ffn(y, up, down, b, lora=None, ids=None):
    def project(z, w, i):
        out = z @ w.mT
        if lora is not None:
            a, bb, al = lora[i]  # the unrotated adapter meets the unrotated activations
            x = _rotate(z, b)
            for n in range(len(al)):
                at = ids == n
                out[at] += x[at] @ a[n].double().mT @ bb[n].double().mT * float(al[n])
        return out

    u = project(_quantized(_rotate(y, b)), up, 0)
    u = (u * torch.special.ndtr(u)).float().to(torch.bfloat16).double()
    return project(_quantized(_rotate(u, b)), down, 1)


def _inputs(t, hid, seed, mods=True, post=True, segments=3):
    g = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(s, generator=g)

    c = dict(x=randn(t, hid).to(torch.bfloat16), r=randn(t, hid).to(torch.bfloat16), nw=torch.rand(hid, generator=g) + 0.5)
    c["post"] = torch.rand(hid, generator=g) + 0.5 if post else None
    c["gate"], c["scale"], c["shift"] = ((randn(segments, hid) * 0.5 for _ in range(3)) if mods else (None, None, None))
    c["seg"], c["rs"] = torch.randint(0, segments, (t,), generator=g), 0.75 if post else 1.0
    return g, c


def _mods(c):
    if c["gate"] is None:
        return {}
    return dict(gate=c["gate"].cuda(), scale=c["scale"].cuda(), shift=c["shift"].cuda(), segment=c["seg"].int().cuda())


def _close(y, ref, bound=2.0 ** -7):
    assert torch.isfinite(y).all()
    assert float((y.double().cpu() - ref).norm() / ref.norm()) < bound


def _check_h(h, ref):
    assert float((h.double().cpu() - ref).abs().max()) <= 2.0 ** -8 * float(ref.abs().max())


@pytest.mark.parametrize("t", [1, 7, 32, 33, 150])
@pytest.mark.parametrize("mods,post", [(True, True), (True, False), (False, True)])
def test_dense_block(ffn, ops, t, mods, post):
    hid, f, b = 256, 640, 64
    g, c = _inputs(t, hid, t, mods, post)
    up, down = (ops.pack_weights((torch.randn(s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))
    layer = ffn.FFN(up, down, c["nw"].cuda(), b, post_weight=None if c["post"] is None else c["post"].cuda(),
                    residual_scale=c["rs"])
    y, h = layer(c["x"].cuda(), c["r"].cuda(), **_mods(c))
    layer.check()
    want, z = _stream(c)
    _check_h(h, want)
    _close(y, _ffn(z, _weight(up.i4_codes, up.i4_scales), _weight(down.i4_codes, down.i4_scales), b))
    y2, _ = layer(y, h, **_mods(c))  # chains
    assert y2.shape == y.shape and torch.isfinite(y2).all()


@pytest.mark.parametrize("t", [1, 5, 32, 33, 200, 2100])
def test_dense_with_adapters(ffn, ops, t):
    hid, f, b, count, rank = 256, 640, 64, 4, 8
    g, c = _inputs(t, hid, 10 + t, mods=t != 5)
    up, down = (ops.pack_weights((torch.randn(s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))

    def adapters(n, k):
        a = (torch.randn((count, rank, k), generator=g) * k ** -0.5).to(torch.bfloat16)
        return a, (torch.randn((count, n, rank), generator=g) * 0.2).to(torch.bfloat16), torch.rand(count, generator=g) + 0.5

    lora = [adapters(f, hid), adapters(hid, f)]
    packed = [ops.pack_lowrank(a.cuda(), bb.cuda(), al.cuda(), b) for a, bb, al in lora]
    layer = ffn.FFN(up, down, c["nw"].cuda(), b, post_weight=c["post"].cuda(), residual_scale=c["rs"],
                    up_adapters=packed[0], down_adapters=packed[1])
    ids = torch.randint(-1, count, (t,), generator=g)
    y, _ = layer(c["x"].cuda(), c["r"].cuda(), **_mods(c), adapters=ids.int().cuda())
    layer.check()
    _, z = _stream(c)
    ws = _weight(up.i4_codes, up.i4_scales), _weight(down.i4_codes, down.i4_scales)
    _close(y, _ffn(z, *ws, b, lora, ids), 2.0 ** -6)
    plain = ffn.FFN(up, down, c["nw"].cuda(), b, post_weight=c["post"].cuda(), residual_scale=c["rs"])
    y0, _ = plain(c["x"].cuda(), c["r"].cuda(), **_mods(c))
    assert torch.equal(layer(c["x"].cuda(), c["r"].cuda(), **_mods(c))[0], y0)  # no token's adapters named
    _close(layer(c["x"].cuda(), c["r"].cuda(), **_mods(c), adapters=torch.full_like(ids, -1).int().cuda())[0], _ffn(z, *ws, b))


@pytest.mark.parametrize("t", [1, 6, 40, 300])
@pytest.mark.parametrize("rule", [dict(), dict(score=1, route_scale=2.5), dict(score=1, bias=True, groups=4, top_groups=2),
                                  dict(bias=True, renormalize=False), dict(groups=2, top_groups=1, group_best=1)])
def test_experts(ffn, ops, t, rule):
    hid, f, b, e, k = 256, 384, 64, 8, 2
    g, c = _inputs(t, hid, 100 + t)
    up, down = (ops.pack_experts((torch.randn((e,) + s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))
    router = torch.randn((e, hid), generator=g) * 0.3
    rule = dict(rule)
    bias = torch.randn(e, generator=g) * 0.2 if rule.pop("bias", False) else None
    layer = ffn.MoEFFN(router.cuda(), up, down, k, c["nw"].cuda(), b, bias=None if bias is None else bias.cuda(),
                       post_weight=c["post"].cuda(), residual_scale=c["rs"], **rule)
    y, h = layer(c["x"].cuda(), c["r"].cuda(), **_mods(c))
    layer.check()
    want, z = _stream(c)
    _check_h(h, want)
    # the choice on the layer's own logits (FP32), its rule in float64
    logits = layer.logits(h).double().cpu()
    p = torch.sigmoid(logits) if rule.get("score") else torch.softmax(logits, 1)
    key = p if bias is None else p + bias.double()
    groups, size = rule.get("groups", 1), e // rule.get("groups", 1)
    if groups > 1:
        best = key.view(t, groups, size).topk(min(rule.get("group_best", 2), size), 2).values.sum(2)
        kept = best.topk(rule["top_groups"], 1).indices
        open_ = torch.zeros((t, groups), dtype=torch.bool).scatter(1, kept, True).repeat_interleave(size, 1)
        key = torch.where(open_, key, -torch.inf)
    chosen = key.topk(k, 1).indices
    w = p.gather(1, chosen)
    if rule.get("renormalize", True):
        w = w / w.sum(1, keepdim=True)
    w = w * rule.get("route_scale", 1.0)
    ref = torch.zeros((t, hid), dtype=torch.float64)
    for i in range(e):
        tok, slot = (chosen == i).nonzero(as_tuple=True)
        if len(tok):
            out = _ffn(z[tok], _weight(up.i4_codes[i], up.i4_scales[i]), _weight(down.i4_codes[i], down.i4_scales[i]), b)
            ref.index_add_(0, tok, out * w[tok, slot, None])
    _close(y, ref)


@pytest.mark.parametrize("t,e,k", [(1, 8, 2), (40, 8, 1), (300, 16, 2), (300, 16, 3), (700, 8, 4), (50, 40, 8)])
def test_the_default_rule_is_topk_softmax_and_a_weighted_sum(ffn, ops, t, e, k):
    """Routing and the sum by torch operations give the same bits."""
    hid, b = 256, 64
    g, c = _inputs(t, hid, 7 * t + k, mods=False, post=False)
    up, down = (ops.pack_experts((torch.randn((e,) + s, generator=g) * 0.05).cuda(), b) for s in ((256, hid), (hid, 256)))
    layer = ffn.MoEFFN((torch.randn((e, hid), generator=g) * 0.3).cuda(), up, down, k, c["nw"].cuda(), b)
    x, r = c["x"].cuda(), c["r"].cuda()
    y, h = layer(x, r)
    top = layer.logits(h).topk(k, dim=1)
    weights = torch.softmax(top.values, dim=1)
    rows, w, token, offsets = layer.route(h)
    expert, order = top.indices.flatten().sort(stable=True)
    assert torch.equal(w, weights) and torch.equal(token, order // k) and rows.dtype == token.dtype == torch.int64
    assert torch.equal(order[rows.flatten()], torch.arange(t * k, device="cuda"))
    a, _ = ops.add_rmsnorm_quant(x, r, layer.norm_weight, layer.eps, b)
    a = ops.int8_act(a.i8_codes[token], a.row_scale[token])
    u = ops.qgemm_grouped(a, up, offsets, ops.EPI_GELU)
    q = ops.hadamard_quant(u, b, ops.MODE_INT8, out=ops.QActTensors(*u.shape, u.device, nvfp4=False))
    d = ops.qgemm_grouped(q, down, offsets, out_f32=True)
    assert torch.equal(y, (d[rows] * weights.unsqueeze(-1)).sum(1).to(torch.bfloat16))


def test_more_choices_than_the_kernel_takes(ffn, ops):
    t, hid, b, e, k = 20, 128, 16, 40, 36
    g, c = _inputs(t, hid, 1, mods=False, post=False)
    up, down = (ops.pack_experts((torch.randn((e,) + s, generator=g) * 0.05).cuda(), b) for s in ((128, hid), (hid, 128)))
    layer = ffn.MoEFFN((torch.randn((e, hid), generator=g) * 0.3).cuda(), up, down, k, had_block=b)
    y, _ = layer(c["x"].cuda(), c["r"].cuda())
    assert torch.isfinite(y).all() and layer.route(c["x"].cuda())[0].shape == (t, k)


@pytest.mark.parametrize("t", [1, 33])
def test_blocks_in_a_graph(ffn, ops, t):
    """A dense block with adapters and a routed one behind it, captured, on new inputs."""
    hid, f, b, e = 256, 384, 64, 4
    g, c = _inputs(t, hid, 3)
    up, down = (ops.pack_weights((torch.randn(s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))
    ups, downs = (ops.pack_experts((torch.randn((e,) + s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))
    lora = ops.pack_lowrank((torch.randn((2, 16, hid), generator=g) * 0.06).to(torch.bfloat16).cuda(),
                            (torch.randn((2, f, 16), generator=g) * 0.2).to(torch.bfloat16).cuda(), None, b)
    dense = ffn.FFN(up, down, c["nw"].cuda(), b, post_weight=c["post"].cuda(), up_adapters=lora)
    moe = ffn.MoEFFN(torch.randn((e, hid), generator=g).cuda(), ups, downs, 2, c["nw"].cuda(), b, score=ops.SCORE_SIGMOID,
                     post_weight=c["post"].cuda())
    ids, mods = torch.randint(-1, 2, (t,), generator=g).int().cuda(), _mods(c)
    x, r = c["x"].cuda(), c["r"].cuda()

    def blocks():
        y, h = dense(x, r, **mods, adapters=ids)
        return moe(y, h, **mods)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blocks()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h = blocks()
    for i in range(2):
        x.copy_(torch.randn((t, hid), generator=g).to(torch.bfloat16))
        ids.fill_(i)
        graph.replay()
        got = y.clone(), h.clone()
        want = blocks()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dense.check(), moe.check()


def test_refusals(ffn, ops):
    hid, f, b = 128, 256, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    up, down = (ops.pack_weights(torch.randn(s, generator=g, device="cuda"), b) for s in ((f, hid), (hid, f)))
    lora = ops.pack_lowrank(torch.zeros((1, 16, hid), dtype=torch.bfloat16, device="cuda"),
                            torch.zeros((1, f, 16), dtype=torch.bfloat16, device="cuda"), None, b)
    with pytest.raises(ValueError):
        ffn.FFN(up, down, down_adapters=lora)
    x = torch.zeros((3, hid), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ffn.FFN(up, down, had_block=b)(x, adapters=torch.zeros(3, dtype=torch.int32, device="cuda"))
    layer = ffn.FFN(up, down, had_block=b, up_adapters=lora)
    with pytest.raises(ValueError):
        layer(x, adapters=torch.zeros(2, dtype=torch.int32, device="cuda"))
    layer(x, adapters=torch.ones(3, dtype=torch.int32, device="cuda"))  # there is one adapter
    with pytest.raises(RuntimeError):
        layer.check()
    ups, downs = (ops.pack_experts(torch.randn((4,) + s, generator=g, device="cuda"), b) for s in ((f, hid), (hid, f)))
    moe = ffn.MoEFFN(torch.zeros((4, hid), device="cuda"), ups, downs, 2, had_block=b, normed_router=True)
    with pytest.raises(ValueError):
        moe(x, x, shift=torch.zeros(hid, device="cuda"))
    moe(x, x, gate=torch.ones(hid, device="cuda"))
    with pytest.raises(RuntimeError):
        ffn.MoEFFN(torch.zeros((4, hid), device="cuda"), ups, downs, 2, had_block=b, groups=3)(x)
