"""Feed-forward layers of a transformer block on the INT8 x INT4 path, from one token to a whole video.

Both take a block's branch output and its residual stream and return this layer's branch output and the new
stream, so that layers chain without a separate addition:

    y, h = layer(x, residual)        # h = x + residual,  y = down(GELU(up(norm(h))))

``FFN`` is the dense layer (the few-row product for up to 32 tokens, the GEMM above), ``MoEFFN`` a mixture of
experts whose row counts stay on the device.  Neither synchronises with the host.  Both run on the current stream and
take their buffers from torch's allocator for the call, so that calls on different streams, from different threads or
captured into CUDA graphs do not share any.

The products' waits are bounded.  One that runs out leaves its output unfinished and records that in the layer's
``err`` word; ``layer.check()`` waits for the stream and raises ``SixbitError`` then.
"""
from __future__ import annotations

import torch

from . import ops


class _Layer:
    def check(self, stream=None) -> None:
        """Waits for `stream` (None: the current one) and raises if a product of this layer failed on the GPU since the
        last check."""
        ops.check_err(self.err, type(self).__name__, stream)


class FFN(_Layer):
    """up [F, H], down [H, F]: ops.pack_weights results with this had_block; norm_weight: float32 [H] or None."""

    def __init__(self, up: ops.PackedWeights, down: ops.PackedWeights, norm_weight=None, had_block: int = 64,
                 eps: float = 1e-6):
        if (up.n, up.k) != (down.k, down.n):
            raise ValueError(f"up [{up.n}, {up.k}] and down [{down.n}, {down.k}] do not chain")
        self.up, self.down, self.norm_weight, self.had_block, self.eps = up, down, norm_weight, had_block, eps
        self.err = torch.zeros(1, dtype=torch.int32, device=up.i4_codes.device)

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        a, h = ops.add_rmsnorm_quant(x, residual, self.norm_weight, self.eps, self.had_block)
        if a.m == 0:
            return torch.empty_like(h), h
        if a.m <= ops.QGEMV_MAX_ROWS:
            def product(act, w, epilogue):
                return ops.qgemv(act, w, epilogue, err=self.err)
        else:
            # The GEMM expands its weights here first.  A buffer of the call's own: one shared with calls on other
            # streams, or with a captured graph, would be overwritten while it is read.
            ws = torch.empty(max(ops.qgemm_workspace_bytes(w.n, w.k) for w in (self.up, self.down)),
                             dtype=torch.uint8, device=h.device)

            def product(act, w, epilogue):
                return ops.qgemm(act, None, w, ops.MODE_INT8, epilogue, err=self.err, ws=ws)
        u = product(a, self.up, ops.EPI_GELU)
        q = ops.hadamard_quant(u, self.had_block, ops.MODE_INT8, out=ops.QActTensors(*u.shape, u.device, nvfp4=False))
        return product(q, self.down, ops.EPI_NONE), h


class MoEFFN(_Layer):
    """router [E, H]; up [E, F, H], down [E, H, F]: ops.pack_experts results with this had_block.

    Each token goes to the top_k experts of softmax(router h), or with normed_router of softmax(router norm(h)), as
    a pre-norm block trains it (norm_weight included); their outputs are summed with the probabilities renormalised
    over those experts.  The router reads the new stream h in bf16, in FP32."""

    def __init__(self, router: torch.Tensor, up: ops.Int4Weights, down: ops.Int4Weights, top_k: int, norm_weight=None,
                 had_block: int = 64, eps: float = 1e-6, normed_router: bool = False):
        if up.experts is None or up.experts != down.experts or (up.n, up.k) != (down.k, down.n):
            raise ValueError("up [E, F, H] and down [E, H, F] of the same experts expected")
        if tuple(router.shape) != (up.experts, up.k) or not 1 <= top_k <= up.experts:
            raise ValueError(f"router [{up.experts}, {up.k}] and 1 <= top_k <= {up.experts} expected")
        self.router, self.up, self.down, self.top_k = router.float(), up, down, top_k
        self.norm_weight, self.had_block, self.eps, self.normed_router = norm_weight, had_block, eps, normed_router
        if normed_router and norm_weight is not None:
            self.router = self.router * norm_weight
        self.ids = torch.arange(up.experts + 1, device=router.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=up.i4_codes.device)

    def route(self, h: torch.Tensor):
        """(row of each token's choices [T, k], weights [T, k], token of each row [T k], offsets int32 [E + 1]): the
        T k rows are sorted by expert, rows of one expert by token."""
        h = h.float()
        logits = h @ self.router.mT
        if self.normed_router:  # (the norm's row factor comes out of the product, its weight stands in the router)
            logits *= torch.rsqrt(h.square().mean(1, keepdim=True) + self.eps)
        top = logits.topk(self.top_k, dim=1)
        weights = torch.softmax(top.values, dim=1)
        expert, order = top.indices.flatten().sort(stable=True)
        offsets = torch.searchsorted(expert, self.ids, out_int32=True)
        rows = torch.empty_like(order)
        rows[order] = torch.arange(order.numel(), device=order.device)
        return rows.view_as(weights), weights, order // self.top_k, offsets

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None):
        a, h = ops.add_rmsnorm_quant(x, residual, self.norm_weight, self.eps, self.had_block)
        if a.m == 0:
            return torch.empty_like(h), h
        rows, weights, token, offsets = self.route(h)
        a = ops.int8_act(a.i8_codes[token], a.row_scale[token])
        u = ops.qgemm_grouped(a, self.up, offsets, ops.EPI_GELU, err=self.err)
        q = ops.hadamard_quant(u, self.had_block, ops.MODE_INT8, out=ops.QActTensors(*u.shape, u.device, nvfp4=False))
        d = ops.qgemm_grouped(q, self.down, offsets, out_f32=True, err=self.err)
        return (d[rows] * weights.unsqueeze(-1)).sum(1).to(torch.bfloat16), h
