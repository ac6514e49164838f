"""The calls around a feed-forward layer's products allocate, and ask of a workspace of the user's, the bytes that the
library names (host checks; nothing is launched)."""
import pytest
import torch
from test_layer_operators_device_cpu import OnGpu, ops  # noqa: F401


@pytest.fixture()
def allocated(ops, monkeypatch):  # noqa: F811
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    def empty(shape, dtype, device, stream):
        if dtype is torch.uint8:
            seen.append(shape[0])
        return OnGpu(shape, dtype)

    monkeypatch.setattr(ops, "_lib", Lib())
    monkeypatch.setattr(ops, "_current_device", lambda: 1, raising=False)
    monkeypatch.setattr(ops, "_current_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(ops, "_empty", empty)
    return seen


def _route(ops, t, e, **kw):  # noqa: F811
    return ops.moe_route(OnGpu((t, e), torch.float32), 1, **kw)


def _lowrank(ops, m, r, **kw):  # noqa: F811
    w = ops.LowRank(OnGpu((2, r, 128), torch.bfloat16), OnGpu((2, 64, r), torch.bfloat16))
    act = ops.int8_act(OnGpu((m, 128), torch.int8), OnGpu((m,), torch.float32))
    return ops.lowrank_add(act, w, OnGpu((m,), torch.int32), **kw)


@pytest.mark.parametrize("call,of,sizes", [
    (_route, "moe_route_workspace_bytes", [(1, 8), (32, 64), (33, 64), (40, 7), (5000, 1024)]),
    (_lowrank, "lowrank_workspace_bytes", [(1, 16), (64, 64), (65, 64), (128, 16), (129, 16), (127, 48), (1003, 128)])])
def test_bytes(ops, allocated, call, of, sizes):  # noqa: F811
    from video_dit_mixed_gb300 import abi
    named = getattr(abi.lib(), "sixbit_" + of)
    for size in sizes:
        want = named(*size)
        assert getattr(ops, of)(*size) == want
        allocated.clear()
        call(ops, *size)
        assert allocated == ([want] if want else [])
        if want:
            allocated.clear()
            call(ops, *size, ws=OnGpu((want,), torch.uint8))
            with pytest.raises(ValueError, match="ws"):
                call(ops, *size, ws=OnGpu((want - 1,), torch.uint8))
            assert not allocated


@pytest.mark.parametrize("call,of,size", [(_route, "_route_workspace_bytes", (300, 16)),
                                          (_lowrank, "_lowrank_workspace_bytes", (300, 16))])
def test_the_number_is_the_librarys(ops, allocated, monkeypatch, call, of, size):  # noqa: F811
    """No second copy of the formula."""
    monkeypatch.setattr(ops, of, lambda a, b: 1_234_560)
    call(ops, *size)
    assert allocated == [1_234_560]
