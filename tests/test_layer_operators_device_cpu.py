"""The calls around a feed-forward layer's products run on the tensors' GPU or not at all (host checks; nothing is launched)."""
from types import SimpleNamespace

import pytest
import torch


class OnGpu:
    """What the binding asks of a tensor, on GPU 1."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, "cuda:1"

    def get_device(self):
        return 1

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1

    def stride(self):
        return ()


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import abi
    abi.lib(build_if_missing=True)
    from video_dit_mixed_gb300 import ops as o
    return o


@pytest.fixture()
def called(ops, monkeypatch):
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append((name, a[-1])) or 0

    monkeypatch.setattr(ops, "_lib", Lib())
    monkeypatch.setattr(ops, "_current_raw_stream", lambda dev: 100 + dev)
    monkeypatch.setattr(ops, "_empty", lambda shape, dtype, device, stream: OnGpu(shape, dtype))
    return seen


def _calls(ops, **kw):
    m, n, k, r = 40, 64, 256, 16
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    act = ops.int8_act(OnGpu((m, k), torch.int8), OnGpu((m,), f32))
    lora = ops.LowRank(OnGpu((2, r, k), bf), OnGpu((2, n, r), bf))
    return [
        lambda: ops.gated_rmsnorm_quant(OnGpu((m, k), bf), gate=OnGpu((k,), f32), **kw),
        lambda: ops.moe_route(OnGpu((m, 8), f32), 2, **kw),
        lambda: ops.moe_combine(OnGpu((m, k), f32), OnGpu((5, 2), i32), OnGpu((5, 2), f32), **kw),
        lambda: ops.lowrank_add(act, lora, OnGpu((m,), i32), **kw),
    ]


def test_another_current_device_is_refused(ops, called, monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: 0, raising=False)
    for call in _calls(ops) + _calls(ops, stream=SimpleNamespace(device_index=1, cuda_stream=7)):
        with pytest.raises(ValueError, match="current device"):
            call()
    assert not called


def test_a_stream_of_another_device_is_refused(ops, called, monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: 1, raising=False)
    for call in _calls(ops, stream=SimpleNamespace(device_index=0, cuda_stream=7)):
        with pytest.raises(ValueError, match="stream"):
            call()
    assert not called


def test_the_tensors_device_and_its_streams_are_taken(ops, called, monkeypatch):
    monkeypatch.setattr(ops, "_current_device", lambda: 1, raising=False)
    for call in _calls(ops) + _calls(ops, stream=SimpleNamespace(device_index=1, cuda_stream=7)):
        call()
    assert [s for _, s in called] == [101] * 4 + [7] * 4


@pytest.mark.parametrize("other", ["weight", "gate", "segment", "residual", "post_weight"])
def test_a_tensor_of_another_device_is_refused(ops, called, monkeypatch, other):
    monkeypatch.setattr(ops, "_current_device", lambda: 1, raising=False)
    shapes = dict(weight=((256,), torch.float32), gate=((256,), torch.float32), segment=((4,), torch.int32),
                  residual=((4, 256), torch.bfloat16), post_weight=((256,), torch.float32))
    t = OnGpu(*shapes[other])
    t.get_device = lambda: 0
    with pytest.raises(ValueError):
        ops.gated_rmsnorm_quant(OnGpu((4, 256), torch.bfloat16), **{other: t})
    assert not called
