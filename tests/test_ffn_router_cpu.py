"""MoEFFN.route on the host, against the definition in float64: the router on the stream, or on its norm."""
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def ffn():
    from video_dit_mixed_gb300 import abi
    abi.lib(build_if_missing=True)
    from video_dit_mixed_gb300 import ffn as f
    return f


def _layer(ffn, router, top_k, **kw):
    e, hid = router.shape
    codes = torch.zeros((e, hid, hid // 2), dtype=torch.uint8)
    w = SimpleNamespace(experts=e, n=hid, k=hid, i4_codes=codes)
    return ffn.MoEFFN(router, w, w, top_k, **kw)


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_route(ffn, weight, normed):
    t, hid, e, k, eps = 200, 128, 7, 2, 1e-3
    g = torch.Generator().manual_seed(1)
    router = torch.randn((e, hid), generator=g)
    nw = torch.exp(torch.randn(hid, generator=g)) if weight else None
    h = (torch.randn((t, hid), generator=g) * torch.exp(2 * torch.randn((t, 1), generator=g))).to(torch.bfloat16)
    kw = dict(normed_router=True) if normed else {}
    rows, weights, token, offsets = _layer(ffn, router, k, norm_weight=nw, eps=eps, **kw).route(h)

    y = h.double()
    if normed:
        y = y / (y.square().mean(1, keepdim=True) + eps).sqrt() * (1.0 if nw is None else nw.double())
    top = (y @ router.double().mT).topk(k, dim=1)
    of_row = torch.searchsorted(offsets[1:].long(), rows, right=True)
    assert torch.equal(of_row, top.indices)
    # an error of 2^-23 (hid + 8) of a logit's absolute terms moves a probability by at most half of that
    terms = (y.abs() @ router.double().abs().mT).amax(1, keepdim=True)
    assert torch.all((weights.double() - torch.softmax(top.values, 1)).abs() <= 2.0 ** -23 * ((hid + 8) * terms + 4))
    assert torch.equal(token[rows], torch.arange(t)[:, None].expand(t, k))
    assert offsets.dtype == torch.int32 and int(offsets[0]) == 0 and int(offsets[-1]) == t * k


def test_the_norms_weight_changes_the_choice(ffn):
    """The stream favours expert 0, its norm with this weight expert 1."""
    router = torch.zeros((2, 128))
    router[0, 0], router[1, 1] = 1.0, 1.0
    nw = torch.ones(128)
    nw[0] = 0.1
    h = torch.full((3, 128), 0.5)
    h[:, 0], h[:, 1] = 2.0, 1.0
    for normed, expert in ((False, 0), (True, 1)):
        _, _, _, offsets = _layer(ffn, router, 1, norm_weight=nw, normed_router=normed).route(h.to(torch.bfloat16))
        assert offsets.tolist() == ([0, 3, 3] if expert == 0 else [0, 0, 3])
