"""The device's shared GEMM workspace (ops.workspace; host logic, on CPU tensors)."""
import weakref

import pytest


@pytest.fixture()
def ops(monkeypatch):
    from video_dit_mixed_gb300 import abi
    abi.lib(build_if_missing=True)
    from video_dit_mixed_gb300 import ops as o
    monkeypatch.setattr(o, "_workspaces", {})
    return o


def test_an_outgrown_buffer_stays(ops):
    """Captured graphs and pending launches may still use its address: it must not go back to the allocator."""
    small = ops.workspace(256, 256, "cpu")
    alive, at = weakref.ref(small), small.data_ptr()
    del small
    large = ops.workspace(1024, 256, "cpu")
    assert large.numel() >= ops.qgemm_workspace_bytes(1024, 256) and large.data_ptr() != at
    assert alive() is not None and alive().data_ptr() == at


def test_calls_share_the_largest_buffer(ops):
    a = ops.workspace(1024, 256, "cpu")
    b = ops.workspace(2048, 256, "cpu")
    assert b.numel() > a.numel()
    for n in (256, 1024, 2048):
        assert ops.workspace(n, 256, "cpu").data_ptr() == b.data_ptr()
