"""Feed-forward layers of a transformer block on the INT8 x INT4 path, from one token to a whole video.

Both take a block's branch output and its residual stream and return this layer's branch output and the new
stream, so that layers chain without a separate addition:

    y, h = layer(x, residual)        # h = x + residual,  y = down(GELU(up(norm(h))))

``FFN`` is the dense layer (the few-row product for up to 32 tokens, the GEMM above), ``MoEFFN`` a mixture of
experts whose row counts stay on the device.  A block may norm and gate its branch before it joins the stream and
modulate the norm behind it:

    h = residual_scale residual + gate [post norm](x),  y = down(GELU(up(norm(h) (1 + scale) + shift)))

and ``FFN`` may have low-rank adapters of many requests beside its projections.  Neither synchronises with the host.
Both run on the current stream and take their buffers from torch's allocator for the call, so that calls on different
streams, from different threads or captured into CUDA graphs do not share any.

The products' waits are bounded.  One that runs out leaves its output unfinished and records that in the layer's
``err`` word; ``layer.check()`` waits for the stream and raises ``SixbitError`` then.
"""
from __future__ import annotations

import math

import torch

from . import abi, ops


class _Layer:
    norm_weight = post_weight = None
    residual_scale = 1.0

    def _norm(self, x, residual, gate, scale, shift, segment):
        """(INT8 activations, the new stream h).  The plain norm where nothing of the block's own is asked for."""
        if self.post_weight is None and self.residual_scale == 1.0 and gate is None and scale is None and shift is None:
            return ops.add_rmsnorm_quant(x, residual, self.norm_weight, self.eps, self.had_block)
        return ops.gated_rmsnorm_quant(x, residual, self.norm_weight, self.post_weight, gate, scale, shift, segment,
                                       self.residual_scale, self.eps, self.had_block, err=self.err)

    def check(self, stream=None) -> None:
        """Waits for `stream` (None: the current one) and raises if a product of this layer failed on the GPU since the
        last check."""
        ops.check_err(self.err, type(self).__name__, stream)


class FFN(_Layer):
    """up [F, H], down [H, F]: ops.pack_weights results with this had_block; norm_weight: float32 [H] or None.

    post_weight: float32 [H], a norm of the branch that comes in; residual_scale: of the stream.  up_adapters,
    down_adapters: ops.pack_lowrank results with this had_block (None: that projection has none); a call names the
    tokens' adapters."""

    def __init__(self, up: ops.PackedWeights, down: ops.PackedWeights, norm_weight=None, had_block: int = 64,
                 eps: float = 1e-6, post_weight=None, residual_scale: float = 1.0,
                 up_adapters: ops.LowRank | None = None, down_adapters: ops.LowRank | None = None):
        if (up.n, up.k) != (down.k, down.n):
            raise ValueError(f"up [{up.n}, {up.k}] and down [{down.n}, {down.k}] do not chain")
        for w, a in ((up, up_adapters), (down, down_adapters)):
            if a is not None and (a.n, a.k) != (w.n, w.k):
                raise ValueError(f"adapters of [{a.n}, {a.k}] beside a projection of [{w.n}, {w.k}]")
        self.up, self.down, self.norm_weight, self.had_block, self.eps = up, down, norm_weight, had_block, eps
        self.post_weight, self.residual_scale = post_weight, residual_scale
        self.up_adapters, self.down_adapters = up_adapters, down_adapters
        self.err = torch.zeros(1, dtype=torch.int32, device=up.i4_codes.device)

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None, gate=None, scale=None, shift=None,
                 segment=None, adapters: torch.Tensor | None = None):
        """gate, scale, shift, segment: as ops.gated_rmsnorm_quant takes them.  adapters: int32 [T] on the GPU, each
        token's adapter or -1 (None: no token has one)."""
        if adapters is not None and self.up_adapters is None and self.down_adapters is None:
            raise ValueError("adapters named of a layer that has none")
        a, h = self._norm(x, residual, gate, scale, shift, segment)
        if a.m == 0:
            return torch.empty_like(h), h
        if a.m <= ops.QGEMV_MAX_ROWS:
            def product(act, w, epilogue, **kw):
                return ops.qgemv(act, w, epilogue, err=self.err, **kw)
        else:
            # The GEMM expands its weights here first.  A buffer of the call's own: one shared with calls on other
            # streams, or with a captured graph, would be overwritten while it is read.
            ws = torch.empty(max(ops.qgemm_workspace_bytes(w.n, w.k) for w in (self.up, self.down)),
                             dtype=torch.uint8, device=h.device)

            def product(act, w, epilogue, **kw):
                return ops.qgemm(act, None, w, ops.MODE_INT8, epilogue, err=self.err, ws=ws, **kw)

        def projection(act, w, lowrank, epilogue):
            if lowrank is None or adapters is None:
                return product(act, w, epilogue)
            base = product(act, w, ops.EPI_NONE, out_f32=True)  # (the adapters' sum comes before GELU and the rounding)
            return ops.lowrank_add(act, lowrank, adapters, base, epilogue, err=self.err)

        u = projection(a, self.up, self.up_adapters, ops.EPI_GELU)
        q = ops.hadamard_quant(u, self.had_block, ops.MODE_INT8, out=ops.QActTensors(*u.shape, u.device, nvfp4=False))
        return projection(q, self.down, self.down_adapters, ops.EPI_NONE), h


class MoEFFN(_Layer):
    """router [E, H]; up [E, F, H], down [E, H, F]: ops.pack_experts results with this had_block.

    Each token goes to the top_k experts of softmax(router h), or with normed_router of softmax(router norm(h)), as
    a pre-norm block trains it (norm_weight included); their outputs are summed with the probabilities renormalised
    over those experts.  The router reads the new stream h in bf16, in FP32; where it requires a gradient, y and route()'s
    weights carry one to it (y to nothing else: the quantized products have none).  score, bias (float32 [E]), groups,
    top_groups, group_best, renormalize and route_scale are ops.moe_route's; post_weight and residual_scale are
    FFN's."""

    def __init__(self, router: torch.Tensor, up: ops.Int4Weights, down: ops.Int4Weights, top_k: int, norm_weight=None,
                 had_block: int = 64, eps: float = 1e-6, normed_router: bool = False, score: int = ops.SCORE_SOFTMAX,
                 bias: torch.Tensor | None = None, groups: int = 1, top_groups: int = 1, group_best: int = 2,
                 renormalize: bool = True, route_scale: float = 1.0, post_weight=None, residual_scale: float = 1.0):
        if up.experts is None or up.experts != down.experts or (up.n, up.k) != (down.k, down.n):
            raise ValueError("up [E, F, H] and down [E, H, F] of the same experts expected")
        if tuple(router.shape) != (up.experts, up.k) or not 1 <= top_k <= up.experts:
            raise ValueError(f"router [{up.experts}, {up.k}] and 1 <= top_k <= {up.experts} expected")
        self.router, self.up, self.down, self.top_k = router.float(), up, down, top_k
        self.norm_weight, self.had_block, self.eps, self.normed_router = norm_weight, had_block, eps, normed_router
        self.post_weight, self.residual_scale = post_weight, residual_scale
        if normed_router and norm_weight is not None:
            self.router = self.router * norm_weight
        self.rule = dict(score=score, bias=bias, groups=groups, top_groups=top_groups, group_best=group_best,
                         renormalize=renormalize, scale=route_scale)
        self.plain_rule = score == ops.SCORE_SOFTMAX and bias is None and groups == 1 and renormalize and route_scale == 1.0
        self._check_rule(up.experts)
        self.ids = torch.arange(up.experts + 1, device=router.device)
        self.err = torch.zeros(1, dtype=torch.int32, device=up.i4_codes.device)

    def _check_rule(self, e: int) -> None:
        """Refuses a rule that no call could follow: as ops.moe_route would, but when the layer is built."""
        r = self.rule
        bias, groups, top_groups = r["bias"], r["groups"], r["top_groups"]
        if bias is not None and (tuple(bias.shape) != (e,) or bias.dtype != torch.float32 or not bias.is_contiguous() or
                                 bias.device != self.router.device):
            raise ValueError(f"bias: dense float32 [{e}] on {self.router.device} expected")
        if self.top_k > ops.MAX_TOP_K and not self.plain_rule:
            raise ValueError(f"this rule routes to {ops.MAX_TOP_K} experts at most, not to {self.top_k}")
        if (r["score"] not in (ops.SCORE_SOFTMAX, ops.SCORE_SIGMOID) or r["group_best"] not in (1, 2) or
                not math.isfinite(r["scale"]) or not 1 <= groups <= ops.MAX_GROUPS or e % groups or
                not 1 <= top_groups <= groups or self.top_k > top_groups * (e // groups)):
            raise abi.SixbitError(f"MoEFFN: no rule of routing {self.top_k} of {e} experts: "
                                  + ", ".join(f"{k} {v}" for k, v in r.items() if k != "bias"))

    def logits(self, h: torch.Tensor) -> torch.Tensor:
        """The router's logits [T, E] of the stream h."""
        h = h.float()
        logits = h @ self.router.mT
        if self.normed_router:  # (the norm's row factor comes out of the product, its weight stands in the router)
            logits *= torch.rsqrt(h.square().mean(1, keepdim=True) + self.eps)
        return logits

    def route(self, h: torch.Tensor):
        """(row of each token's choices [T, k], weights [T, k], token of each row [T k], offsets int32 [E + 1]): the
        T k rows are sorted by expert, rows of one expert by token.  On the host the default rule alone."""
        return self._choices(self.logits(h))

    def _choices(self, logits: torch.Tensor):
        if self.top_k <= ops.MAX_TOP_K and logits.is_cuda:
            r = ops.moe_route(logits, self.top_k, **self.rule)
            weights = self._weights(logits, r.experts.long()) if logits.requires_grad else r.weights
            return r.rows.long(), weights, r.token.long(), r.offsets
        if not self.plain_rule:
            raise ValueError(f"this rule routes on the GPU, to {ops.MAX_TOP_K} experts at most")
        top = logits.topk(self.top_k, dim=1)
        weights = torch.softmax(top.values, dim=1)
        expert, order = top.indices.flatten().sort(stable=True)
        offsets = torch.searchsorted(expert, self.ids, out_int32=True)
        rows = torch.empty_like(order)
        rows[order] = torch.arange(order.numel(), device=order.device)
        return rows.view_as(weights), weights, order // self.top_k, offsets

    def _weights(self, logits: torch.Tensor, experts: torch.Tensor) -> torch.Tensor:
        """The chosen experts' weights by torch operations, which carry a gradient to the router."""
        chosen = logits.gather(1, experts)
        sigmoid = self.rule["score"] == ops.SCORE_SIGMOID
        if self.rule["renormalize"]:  # (the logarithms of sigmoid scores: their softmax is the scores over their sum)
            w = torch.softmax(torch.nn.functional.logsigmoid(chosen) if sigmoid else chosen, dim=1)
        else:
            w = torch.sigmoid(chosen) if sigmoid else torch.softmax(logits, dim=1).gather(1, experts)
        return w if self.rule["scale"] == 1.0 else w * self.rule["scale"]

    def __call__(self, x: torch.Tensor, residual: torch.Tensor | None = None, gate=None, scale=None, shift=None,
                 segment=None):
        """gate, scale, shift, segment: as ops.gated_rmsnorm_quant takes them (no scale or shift with normed_router)."""
        if self.normed_router and (scale is not None or shift is not None):
            raise ValueError("a router on the norm's output has no modulation")
        a, h = self._norm(x, residual, gate, scale, shift, segment)
        if a.m == 0:
            return torch.empty_like(h), h
        fused = False
        if getattr(self.route, "__func__", None) is not _ROUTE:  # (another's: a subclass's, or one set in its place)
            rows, weights, token, offsets = self.route(h)
        else:
            logits = self.logits(h)
            fused = self.top_k <= ops.MAX_TOP_K and not logits.requires_grad
            if fused:
                _, weights, rows, token, offsets = ops.moe_route(logits, self.top_k, **self.rule)
            else:
                rows, weights, token, offsets = self._choices(logits)
        a = ops.int8_act(a.i8_codes[token], a.row_scale[token])
        u = ops.qgemm_grouped(a, self.up, offsets, ops.EPI_GELU, err=self.err)
        q = ops.hadamard_quant(u, self.had_block, ops.MODE_INT8, out=ops.QActTensors(*u.shape, u.device, nvfp4=False))
        d = ops.qgemm_grouped(q, self.down, offsets, out_f32=True, err=self.err)
        if fused:
            return ops.moe_combine(d, rows, weights, err=self.err), h
        return (d[rows] * weights.unsqueeze(-1)).sum(1).to(torch.bfloat16), h


_ROUTE = MoEFFN.route
