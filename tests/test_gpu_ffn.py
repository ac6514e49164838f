"""The feed-forward layers against the same layer in 64 bits on the packed weights.

The reference quantizes its own activations in float64; a code can land on the other side of a rounding tie and the
intermediate u is rounded to bf16 on both sides, so y agrees in norm only: u's roundings are 2^-9 each, a flipped code
moves one term of a sum of hundreds by 1/127 of its row's largest, and the output's own rounding is 2^-9.  Bound: 2^-7.
"""
import numpy as np
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
    return (y.view(-1, b) @ h / b ** 0.5).view_as(y)


def _quantized(y):
    s = y.abs().amax(1, keepdim=True) / 127
    return torch.round(y / s.clamp(min=1e-300)) * s


def _weight(codes, scales):
    """[N, K] float64 (rotated) from INT4 codes [N, K/2] and scales [K/128, N]."""
    c = codes.cpu().to(torch.int16)
    q = (torch.stack((c & 15, c >> 4), -1).flatten(1) ^ 8) - 8
    return q.double() * scales.cpu().double().repeat_interleave(128, 0).mT


def _ref(h, norm_w, up, down, b):
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * norm_w
    u = _quantized(_rotate(y, b)) @ up.mT
    u = (u * torch.special.ndtr(u)).float().to(torch.bfloat16).double()
    return _quantized(_rotate(u, b)) @ down.mT


def _inputs(t, hid, seed):
    g = torch.Generator().manual_seed(seed)
    x, r = (torch.randn((t, hid), generator=g).to(torch.bfloat16) for _ in range(2))
    return g, x, r, torch.rand(hid, generator=g) + 0.5


def _close(y, ref):
    assert torch.isfinite(y).all()
    assert float((y.double().cpu() - ref).norm() / ref.norm()) < 2.0 ** -7


@pytest.mark.parametrize("t", [1, 2, 7, 32, 33, 150])
def test_dense(ffn, ops, t):
    hid, f, b = 256, 640, 64
    g, x, r, nw = _inputs(t, hid, t)
    up, down = (ops.pack_weights((torch.randn(s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))
    layer = ffn.FFN(up, down, nw.cuda(), b)
    y, h = layer(x.cuda(), r.cuda())
    assert torch.equal(h.cpu(), (x.float() + r.float()).to(torch.bfloat16))
    ref = _ref(x.double() + r.double(), nw.double(), _weight(up.i4_codes, up.i4_scales),
               _weight(down.i4_codes, down.i4_scales), b)
    _close(y, ref)
    none = torch.empty((0, hid), dtype=torch.bfloat16, device="cuda")
    assert all(v.shape == (0, hid) for v in layer(none, none.clone()))
    y2, h2 = layer(y, h)  # chains
    assert y2.shape == y.shape and torch.equal(h2.cpu(), (y.float() + h.float()).to(torch.bfloat16).cpu())


@pytest.mark.parametrize("t,e,k", [(1, 4, 2), (5, 8, 2), (12, 3, 1), (40, 8, 2), (300, 4, 2), (700, 16, 3)])
def test_experts(ffn, ops, t, e, k):
    hid, f, b = 256, 384, 64
    g, x, r, nw = _inputs(t, hid, 100 + t)
    up, down = (ops.pack_experts((torch.randn((e,) + s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))
    router = torch.randn((e, hid), generator=g) * 0.3
    layer = ffn.MoEFFN(router.cuda(), up, down, k, nw.cuda(), b)
    y, h = layer(x.cuda(), r.cuda())
    hb = h.float().cpu()
    top = (h.float() @ router.cuda().mT).topk(k, dim=1)
    probs, chosen = torch.softmax(top.values, 1).double().cpu(), top.indices.cpu()
    ref = torch.zeros((t, hid), dtype=torch.float64)
    full = x.double() + r.double()
    for i in range(e):
        tok, slot = (chosen == i).nonzero(as_tuple=True)
        if len(tok):
            out = _ref(full[tok], nw.double(), _weight(up.i4_codes[i], up.i4_scales[i]),
                       _weight(down.i4_codes[i], down.i4_scales[i]), b)
            ref.index_add_(0, tok, out * probs[tok, slot, None])
    assert torch.equal(hb, (x.float() + r.float()).to(torch.bfloat16).float())
    _close(y, ref)


def test_routing(ffn, ops):
    e, hid, t, k = 5, 128, 64, 2
    g = torch.Generator(device="cuda").manual_seed(1)
    router = torch.randn((e, hid), generator=g, device="cuda")
    w = ops.pack_experts(torch.randn((e, hid, hid), generator=g, device="cuda"), 16)
    layer = ffn.MoEFFN(router, w, w, k, had_block=16)
    h = torch.randn((t, hid), generator=g, device="cuda").to(torch.bfloat16)
    rows, weights, token, offsets = layer.route(h)
    top = (h.float() @ router.mT).topk(k, dim=1).indices
    assert offsets.dtype == torch.int32 and int(offsets[0]) == 0 and int(offsets[-1]) == t * k
    of_row = torch.searchsorted(offsets[1:].long(), rows, right=True)
    assert torch.equal(of_row, top) and torch.equal(token[rows], torch.arange(t, device="cuda")[:, None].expand(t, k))
    assert torch.allclose(weights.sum(1), torch.ones(t, device="cuda"))


def test_refusals(ffn, ops):
    g = torch.Generator(device="cuda").manual_seed(1)
    w = ops.pack_experts(torch.randn((2, 256, 128), generator=g, device="cuda"), 16)
    d = ops.pack_experts(torch.randn((2, 128, 256), generator=g, device="cuda"), 16)
    router = torch.zeros((2, 128), device="cuda")
    for bad in (lambda: ffn.MoEFFN(router, w, w, 1), lambda: ffn.MoEFFN(router, w, d, 3),
                lambda: ffn.MoEFFN(router[:1], w, d, 1)):
        with pytest.raises(ValueError):
            bad()
    p = ops.pack_weights(torch.randn((256, 128), generator=g, device="cuda"), 16)
    with pytest.raises(ValueError):
        ffn.FFN(p, p)
