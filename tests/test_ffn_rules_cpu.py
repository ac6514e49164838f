"""MoEFFN refuses a rule of routing that no call could use when it is built, not at its first call."""
import math
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def ffn():
    from video_dit_mixed_gb300 import abi
    abi.lib(build_if_missing=True)
    from video_dit_mixed_gb300 import ffn as f
    return f


def _layer(ffn, e=8, k=2, **kw):
    w = SimpleNamespace(experts=e, n=16, k=16, i4_codes=torch.zeros((e, 16, 8), dtype=torch.uint8))
    return ffn.MoEFFN(torch.zeros((e, 16)), w, w, k, **kw)


@pytest.mark.parametrize("kw", [dict(), dict(score=1), dict(groups=4, top_groups=1), dict(groups=4, top_groups=4, group_best=1),
                                dict(groups=8, top_groups=2), dict(bias=torch.zeros(8)), dict(route_scale=2.5),
                                dict(renormalize=False), dict(e=40, k=36), dict(e=64, k=32, score=1)])
def test_rules_that_there_are(ffn, kw):
    _layer(ffn, **kw)


@pytest.mark.parametrize("bias", [torch.zeros(7), torch.zeros((8, 1)), torch.zeros(8, dtype=torch.float64),
                                  torch.zeros(8, dtype=torch.bfloat16), torch.zeros(8, device="meta"), torch.zeros(16)[::2]])
def test_a_bias_of_the_wrong_kind(ffn, bias):
    with pytest.raises(ValueError, match="bias"):
        _layer(ffn, bias=bias)


@pytest.mark.parametrize("kw", [dict(score=2), dict(groups=3), dict(groups=0), dict(groups=4, top_groups=0),
                                dict(groups=4, top_groups=5), dict(k=3, groups=4, top_groups=1), dict(group_best=3),
                                dict(group_best=0), dict(route_scale=math.nan), dict(route_scale=math.inf),
                                dict(e=128, groups=64, top_groups=2)])
def test_numbers_that_the_call_refuses(ffn, kw):
    """The error is the call's."""
    with pytest.raises(RuntimeError):
        _layer(ffn, **kw)


@pytest.mark.parametrize("kw", [dict(score=1), dict(route_scale=2.0), dict(renormalize=False), dict(groups=2, top_groups=2)])
def test_more_choices_than_the_rule_can_make(ffn, kw):
    with pytest.raises(ValueError):
        _layer(ffn, 40, 36, **kw)
    _layer(ffn, 40, 36)
