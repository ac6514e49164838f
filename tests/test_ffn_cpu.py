"""The feed-forward layers' host side: which buffers they hand to the products (the calls themselves are stood in for)."""
from types import SimpleNamespace

import pytest
import torch


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import abi
    abi.lib(build_if_missing=True)
    from video_dit_mixed_gb300 import ops as o
    return o


def _dense_layer(n, k):
    return SimpleNamespace(n=n, k=k, i4_codes=torch.zeros((n, k // 2), dtype=torch.uint8))


@pytest.fixture()
def calls(ops, monkeypatch):
    """ffn.FFN on the host: the products are recorded as (name, weights, arguments)."""
    seen = []

    def product(name):
        def call(act, *args, **kw):
            w = args[1] if name == "qgemm" else args[0]
            seen.append((name, w, kw))
            return torch.zeros((act.m, w.n), dtype=torch.bfloat16)
        return call

    def norm(x, *_, **__):
        return SimpleNamespace(m=x.shape[0], k=x.shape[1]), x

    def quant(u, *_, **__):
        return SimpleNamespace(m=u.shape[0], k=u.shape[1])

    monkeypatch.setattr(ops, "add_rmsnorm_quant", norm)
    monkeypatch.setattr(ops, "hadamard_quant", quant)
    monkeypatch.setattr(ops, "qgemm", product("qgemm"))
    monkeypatch.setattr(ops, "qgemv", product("qgemv"))
    return seen


def test_dense_layer_shares_no_workspace(ops, calls, monkeypatch):
    """Above the few-row product's limit every call brings its own workspace, large enough for both products."""
    from video_dit_mixed_gb300 import ffn
    monkeypatch.setattr(ops, "_workspaces", {})
    up, down = _dense_layer(640, 256), _dense_layer(256, 640)
    layer, other = ffn.FFN(up, down), ffn.FFN(up, down)
    x = torch.zeros((ops.QGEMV_MAX_ROWS + 1, 256), dtype=torch.bfloat16)
    for f in (layer, layer, other):
        f(x)
    assert [n for n, _, _ in calls] == ["qgemm"] * 6 and not ops._workspaces
    ws = [kw.get("ws") for _, _, kw in calls]
    for (_, w, _), b in zip(calls, ws):
        assert b is not None and b.numel() * b.element_size() >= ops.qgemm_workspace_bytes(w.n, w.k)
    spans = [(b.data_ptr(), b.data_ptr() + b.numel()) for b in ws[::2]]  # (all kept alive in `calls`)
    for i, (a, b) in enumerate(spans):
        assert all(b <= c or d <= a for c, d in spans[i + 1:])


def test_dense_layer_of_few_rows_needs_none(ops, calls):
    from video_dit_mixed_gb300 import ffn
    layer = ffn.FFN(_dense_layer(640, 256), _dense_layer(256, 640))
    layer(torch.zeros((ops.QGEMV_MAX_ROWS, 256), dtype=torch.bfloat16))
    assert [n for n, _, _ in calls] == ["qgemv"] * 2


@pytest.mark.parametrize("t", [1, 32, 33])
def test_every_product_reports_into_the_layers_word(ops, calls, t):
    from video_dit_mixed_gb300 import ffn
    layer = ffn.FFN(_dense_layer(640, 256), _dense_layer(256, 640))
    layer(torch.zeros((t, 256), dtype=torch.bfloat16))
    assert layer.err.dtype == torch.int32 and layer.err.numel() == 1
    assert [kw.get("err") is layer.err for _, _, kw in calls] == [True, True]
