"""A route() of a subclass, of an instance or of a patched class is the one that MoEFFN uses."""
import pytest
import torch
from test_gpu_ffn_router_gradient import _layer, ffn, ops  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("trained", [False, True])
@pytest.mark.parametrize("how", ["subclass", "instance", "class", "super"])
def test_a_route_of_the_users_own(ffn, ops, monkeypatch, how, trained):  # noqa: F811
    """All tokens to expert 1, weight 0.5."""
    def route(self, h):
        t = h.shape[0]
        i = torch.arange(t, device=h.device)
        offsets = torch.full((9,), t, dtype=torch.int32, device=h.device)
        offsets[:2] = 0
        return i[:, None], torch.full((t, 1), 0.5, device=h.device), i, offsets

    layer, _, x, r, _ = _layer(ffn, ops, 50, k=1, trained=trained)
    want, _ = layer(x, r)
    if how == "subclass":
        layer.__class__ = type("Own", (ffn.MoEFFN,), dict(route=route))
    elif how == "instance":
        layer.route = lambda h: route(layer, h)
    elif how == "class":
        monkeypatch.setattr(ffn.MoEFFN, "route", route)
    else:
        seen = []
        layer.__class__ = type("Seen", (ffn.MoEFFN,), dict(
            route=lambda self, h: seen.append(h.shape) or ffn.MoEFFN.route(self, h)))
        y, _ = layer(x, r)
        assert seen == [x.shape] and torch.equal(y, want)
        return
    y, _ = layer(x, r)
    a, _ = ops.add_rmsnorm_quant(x, r, None, layer.eps, layer.had_block)
    offsets = route(layer, x)[3]
    u = ops.qgemm_grouped(a, layer.up, offsets, ops.EPI_GELU)
    q = ops.hadamard_quant(u, layer.had_block, ops.MODE_INT8, out=ops.QActTensors(*u.shape, u.device, nvfp4=False))
    d = ops.qgemm_grouped(q, layer.down, offsets, out_f32=True)
    assert torch.equal(y, (d * 0.5).to(torch.bfloat16))
