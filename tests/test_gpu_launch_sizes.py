"""Sizes whose shared memory is just below 48 KB without the kernel's own static part, each in a process that has launched
nothing larger before (a larger launch would have raised the kernel's limit for it)."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))

ROUTE = """
import torch
from video_dit_mixed_gb300 import ops
from test_gpu_moe_route import _check, _logits, _ref
t, e, k = 70, {e}, {k}
z, bias = _logits(t, e, e)
r = ops.moe_route(z.cuda(), k, ops.SCORE_SIGMOID, bias=bias.cuda(), groups={groups}, top_groups=3)
_check(r, *_ref(z, k, True, bias, {groups}, 3), e)
"""
LOWRANK = """
import torch
from video_dit_mixed_gb300 import ops
count, m, k, n = {count}, 700, 128, 8
ids = torch.randint(0, count, (m,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
ids[:3] = torch.tensor([0, count - 1, -1], dtype=torch.int32)
a = torch.zeros((count, 16, k), dtype=torch.bfloat16, device="cuda")
a[:, 0, 0] = 1.0
b = torch.zeros((count, n, 16), dtype=torch.bfloat16, device="cuda")
b[:, :, 0] = (torch.arange(count, device="cuda") % 251).to(torch.bfloat16)[:, None]  # whole numbers below 256
x = torch.ones((m, k), dtype=torch.bfloat16, device="cuda")
y = ops.lowrank_add(x, ops.LowRank(a, b), ids.cuda(), out_f32=True)
want = torch.where(ids >= 0, ids % 251, 0).float()
assert torch.equal(y.cpu(), want[:, None].expand(m, n))
"""


def _run(code):
    path = os.pathsep.join([os.path.dirname(HERE), HERE])
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, PYTHONPATH=path), capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("e,k,groups", [(336, 8, 8), (352, 8, 8), (320, 32, 8)])
def test_routing(e, k, groups):
    _run(ROUTE.format(e=e, k=k, groups=groups))


@pytest.mark.parametrize("count", [6128, 6140])
def test_adapters(count):
    _run(LOWRANK.format(count=count))
