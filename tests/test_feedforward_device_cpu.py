"""The feed-forward calls run on the tensors' GPU or not at all (host checks; nothing is launched)."""
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
    return seen


def _calls(ops, **kw):
    m, n, k, e = 4, 64, 256, 2
    act = ops.int8_act(OnGpu((m, k), torch.int8), OnGpu((m,), torch.float32))
    one = ops.Int4Weights(OnGpu((n, k // 2), torch.uint8), OnGpu((k // 128, n), torch.float32))
    many = ops.Int4Weights(OnGpu((e, n, k // 2), torch.uint8), OnGpu((e, k // 128, n), torch.float32))
    y = OnGpu((m, n), torch.bfloat16)
    return [
        lambda: ops.add_rmsnorm_quant(OnGpu((m, k), torch.bfloat16), out=act, **kw),
        lambda: ops.qgemv(act, one, out=y, **kw),
        lambda: ops.qgemm_grouped(act, many, OnGpu((e + 1,), torch.int32), out=y, ws=OnGpu((1 << 16,), torch.uint8), **kw),
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
    assert [s for _, s in called] == [101] * 3 + [7] * 3
