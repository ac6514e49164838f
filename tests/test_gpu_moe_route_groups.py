"""Groups of experts whose keys FP32 holds badly: biases of opposite signs that cancel in a group's sum, and experts taken
out of service by a bias of -infinity, against float64."""
import numpy as np
import pytest
import torch
from test_gpu_moe_route import _check, _check_places, _logits, _ref, ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2, 5, 32])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("large", [30.0, 100.0, 1000.0])
def test_biases_that_cancel(ops, large, sigmoid, size):  # noqa: F811
    """One expert of each group far up, all others far down: a key is held to 2^-24 of the bias, and the groups' sums, below
    2 in size, lie a few such steps apart."""
    groups, top, t, k = 8, 4, 600, 6
    e = groups * size
    g = torch.Generator().manual_seed(int(large) + size)
    step = large * 2.0 ** -24  # (a score of 1/2 or 1/e moves by a quarter or 1/e of its logit)
    z = (torch.randn((t, e), generator=g) * step * (16 if sigmoid else 4 * e)).float()
    bias = torch.full((groups, size), -large)
    bias[torch.arange(groups), torch.randint(0, size, (groups,), generator=g)] = large
    bias = bias.flatten()
    want = _ref(z, k, sigmoid, bias, groups, top)
    r = ops.moe_route(z.cuda(), k, int(sigmoid), bias=bias.cuda(), groups=groups, top_groups=top)
    _check(r, *want, e)


@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("e,k,groups", [(12, 6, 3), (64, 5, 8), (300, 12, 4), (48, 3, 24)])
def test_experts_out_of_service(ops, e, k, groups, sigmoid, best):  # noqa: F811
    """Some, half and nearly all experts at -infinity: groups of them come last, the lower number first among equals."""
    z, bias = _logits(90, e, e + k)
    size = e // groups
    for n in (1, size, e // 2, e - size, e - 1, e):
        b = bias.clone()
        b[torch.randperm(e, generator=torch.Generator().manual_seed(n))[:n]] = -np.inf
        for top in {(groups + 1) // 2, groups}:
            kw = dict(groups=groups, top_groups=top)
            r = ops.moe_route(z.cuda(), k, int(sigmoid), bias=b.cuda(), group_best=best, **kw)
            ex, w = _ref(z, k, sigmoid, b, best=best, **kw)
            assert np.array_equal(r.experts.cpu().numpy(), ex)
            assert np.allclose(r.weights.cpu().numpy(), w, rtol=1e-5, atol=1e-30)
            _check_places(r, e)
