"""pack_experts refuses what it cannot read with a ValueError, whatever assertions are switched off (host only)."""
import pytest
import torch


class OnGpu:
    """A float32 [2, 128, 256] tensor on GPU 0, but for what is given."""

    def __init__(self, dtype=torch.float32, dense=True, dev=0):
        self.shape, self.dtype, self.dense, self.dev = torch.Size((2, 128, 256)), dtype, dense, dev
        self.device = torch.device("cuda", dev) if dev >= 0 else torch.device("cpu")

    def dim(self):
        return 3

    def is_contiguous(self):
        return self.dense

    def stride(self):
        return (128 * 256, 256, 1) if self.dense else (128 * 256, 1, 128)

    def get_device(self):
        return self.dev


@pytest.mark.parametrize("kw", [dict(dtype=torch.bfloat16), dict(dtype=torch.float64), dict(dense=False), dict(dev=-1)])
def test_refusals(kw):
    from video_dit_mixed_gb300 import abi
    abi.lib(build_if_missing=True)
    from video_dit_mixed_gb300 import ops
    with pytest.raises(ValueError, match="dense float32"):
        ops.pack_experts(OnGpu(**kw), 64)
    with pytest.raises(ValueError, match="E, N, K"):
        ops.pack_experts(torch.zeros((128, 256)), 64)
