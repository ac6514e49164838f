"""Performance cases of the quantized feed-forward operators.

Three operators that a quantized feed-forward layer runs next to the rotation,
quantization and GEMM calls, from a single token to a whole video:

``norm``     residual add, root-mean-square norm, optional block-Hadamard
             rotation and per-token INT8 quantization in one call
``gemv``     W4A8 product of 1 to 32 tokens: INT8 codes against INT4 weights
             with one scale per 128 inputs
``experts``  W4A8 product grouped by expert, with ragged row counts on the device

``listed()`` gives the named cases, ``draw(rng)`` more of the same ranges.
``prepare`` makes a case's inputs, ``run`` one pass: in plain torch operations
when ``own`` is false, through the library when it is true.  ``exact`` is the
operators' definition in 64 bits.  All sums are in 32 bits or more; 8-bit
results are returned as the values they stand for.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6
GROUP = 128  # inputs that share one weight scale
MAX_TOKENS = 17776  # 13 x 30 x 45 latent positions and 226 text tokens
MAX_GEMV_TOKENS = 32
MAX_WORK = 2 * MAX_TOKENS * 1920 * 7680  # rows x inputs x outputs of the largest grouped product
MAX_WEIGHTS = 64 * 7680 * 1920  # weights over all experts


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One token of an autoregressive step entering a feed-forward layer of the 2B-shaped model: latency.
        dict(name="norm_1tok", op="norm", m=1, k=1920, had=64, residual=True, weight=True),
        # The text tokens of a prompt.
        dict(name="norm_text", op="norm", m=226, k=1920, had=64, residual=True, weight=True),
        # A block boundary of the 2B-shaped model: every token of a 49-frame video.
        dict(name="norm_video", op="norm", m=17776, k=1920, had=64, residual=True, weight=True),
        # An odd number of wide rows, no branch to add, no rotation (weights packed unrotated elsewhere).
        dict(name="norm_wide_odd", op="norm", m=1003, k=7680, had=0, residual=False, weight=True),
        # Up projection of one token, 2B shapes.
        dict(name="gemv_1tok_up", op="gemv", m=1, n=7680, k=1920, epilogue="gelu", f32=False),
        # Down projection of one token, 5B shapes: few outputs, a long sum.
        dict(name="gemv_1tok_down", op="gemv", m=1, n=3072, k=12288, epilogue="residual", f32=False),
        # Three tokens through a small projection with an odd number of outputs, float output (router or head).
        dict(name="gemv_3tok_odd", op="gemv", m=3, n=1111, k=640, epilogue="none", f32=True),
        # A batch of 32 single tokens, up projection of the 5B shapes.
        dict(name="gemv_32tok_up", op="gemv", m=32, n=12288, k=3072, epilogue="gelu", f32=False),
        # Eight single tokens, two experts each, out of eight.
        dict(name="experts_decode", op="experts", rows=16, experts=8, n=7680, k=1920, skew=0.5, route=1,
             epilogue="gelu", f32=False),
        # The text tokens, two experts each out of 64: most experts have a few rows, some none.
        dict(name="experts_text", op="experts", rows=452, experts=64, n=7680, k=1920, skew=1.0, route=2,
             epilogue="gelu", f32=False),
        # Every video token, two experts each out of eight, up projection.
        dict(name="experts_video_up", op="experts", rows=2 * MAX_TOKENS, experts=8, n=7680, k=1920, skew=0.5,
             route=3, epilogue="gelu", f32=False),
        # One expert per video token, down projection with the residual.
        dict(name="experts_video_down", op="experts", rows=MAX_TOKENS, experts=8, n=1920, k=7680, skew=1.0,
             route=4, epilogue="residual", f32=False),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "gemv", "experts"])
    if op == "norm":
        k = GROUP * _log(rng, 1, 96)
        m = _log(rng, 1, max(1, min(MAX_TOKENS, MAX_TOKENS * 1920 // k)))
        return dict(op=op, m=m, k=k, had=rng.choice([0, 16, 64] + ([256] if k % 256 == 0 else [])),
                    residual=rng.random() < 0.7, weight=rng.random() < 0.7)
    epilogue, f32 = rng.choice(["none", "gelu", "residual"]), rng.random() < 0.3
    if op == "gemv":
        return dict(op=op, m=rng.randint(1, MAX_GEMV_TOKENS), n=_log(rng, 16, 15360), k=GROUP * _log(rng, 1, 96),
                    epilogue=epilogue, f32=f32)
    while True:
        c = dict(op=op, rows=_log(rng, 1, 2 * MAX_TOKENS), experts=_log(rng, 1, 64), n=_log(rng, 64, 7680),
                 k=GROUP * _log(rng, 1, 96), skew=round(rng.uniform(0.0, 1.5), 2), route=rng.randint(0, 9999),
                 epilogue=epilogue, f32=f32)
        if c["rows"] * c["n"] * c["k"] <= MAX_WORK and c["experts"] * c["n"] * c["k"] <= MAX_WEIGHTS:
            return c


def _counts(case):
    """Rows of each expert: shares 1 / rank^skew in an order of the case's own, drawn row by row."""
    rng = random.Random(case["route"])
    share = [1.0 / (r + 1) ** case["skew"] for r in range(case["experts"])]
    rng.shuffle(share)
    counts = [0] * case["experts"]
    for e in rng.choices(range(case["experts"]), weights=share, k=case["rows"]):
        counts[e] += 1
    return counts


def work(case):
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        words = m * k * (2 + (2 + 2 if case["residual"] else 0) + 1) + 4 * m + (4 * k if case["weight"] else 0)
        return {"bytes": words, "flops": m * k * (6 + (int(math.log2(case["had"])) if case["had"] else 0))}
    if case["op"] == "gemv":
        rows, live = case["m"], 1
    else:
        rows, live = case["rows"], sum(c > 0 for c in _counts(case))
    n, k = case["n"], case["k"]
    weights = live * (n * k // 2 + n * (k // GROUP) * 4)
    out = rows * n * (4 if case["f32"] else 2) + (rows * n * 2 if case["epilogue"] == "residual" else 0)
    return {"bytes": weights + rows * (k + 4) + out, "flops": 2 * rows * n * k}


# ------------------------------------------------------------------ inputs --

def _activations(g, m, k, outlier):
    """bf16 Laplace rows with 0.5 % outlier channels, as a transformer block's input has them."""
    u = torch.rand((m, k), generator=g, device="cuda") - 0.5
    x = -torch.sign(u) * torch.log1p(-2.0 * u.abs().clamp(max=0.4999999))
    loud = torch.rand((k,), generator=g, device="cuda") < 0.005
    return torch.where(loud, x * outlier, x).to(torch.bfloat16)


def _int4_weights(g, lead, n, k):
    """INT4 codes [.., n, k/2] (two's-complement nibbles in [-7, 7], even k low) and scales [.., k/128, n]."""
    codes = torch.empty(lead + (n, k // 2), dtype=torch.uint8, device="cuda")
    for c in codes.view(-1, n, k // 2):  # one expert at a time: the draws of a large layer do not fit at once
        q = (torch.randn((n, k), generator=g, device="cuda") * 2.5).round_().clamp_(-7, 7).to(torch.int16) & 15
        c.copy_(q[:, 0::2] | (q[:, 1::2] << 4))
    scales = torch.rand(lead + (k // GROUP, n), generator=g, device="cuda") * 0.01 + 0.005
    return codes, scales


def _int8_rows(g, m, k):
    """INT8 codes [m, k] whose largest is 127 in each row, and the rows' scales."""
    x = torch.randn((m, k), generator=g, device="cuda")
    codes = (x * (127.0 / x.abs().amax(1, keepdim=True))).round_().to(torch.int8)
    return codes, torch.exp(torch.randn((m,), generator=g, device="cuda") * 0.5) * 0.03


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "norm":
        m, k = case["m"], case["k"]
        s["x"] = _activations(g, m, k, 50.0 if case["had"] else 8.0)
        s["res"] = torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16) if case["residual"] else None
        if m > 2:  # a padding token
            s["x"][m // 2] = 0
            if s["res"] is not None:
                s["res"][m // 2] = 0
        s["w"] = torch.rand((k,), generator=g, device="cuda") + 0.5 if case["weight"] else None
        s["rotation"] = _sylvester(case["had"]) if case["had"] else None  # a constant that a program keeps
        return s
    k, n = case["k"], case["n"]
    rows, lead = (case["m"], ()) if case["op"] == "gemv" else (case["rows"], (case["experts"],))
    s["codes"], s["scale"] = _int8_rows(g, rows, k)
    s["w4"], s["w4_scale"] = _int4_weights(g, lead, n, k)
    s["res"] = None
    if case["epilogue"] == "residual":
        s["res"] = torch.randn((rows, n), generator=g, device="cuda").to(torch.bfloat16)
    if case["op"] == "experts":
        counts = _counts(case)
        s["most"] = max(counts)
        s["offsets"] = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    return s


# ------------------------------------------------------------------ a pass --

def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from video_dit_mixed_gb300 import ops

    if s["op"] == "norm":
        a, h = ops.add_rmsnorm_quant(s["x"], s["res"], s["w"], eps=EPS, had_block=s["had"])
        out = {"value": _values(a.i8_codes, a.row_scale), "scale": a.row_scale}
        return dict(out, sum=h) if s["residual"] else out
    a, w = ops.int8_act(s["codes"], s["scale"]), ops.Int4Weights(s["w4"], s["w4_scale"])
    epilogue = {"none": ops.EPI_NONE, "gelu": ops.EPI_GELU, "residual": ops.EPI_RESIDUAL}[s["epilogue"]]
    if s["op"] == "gemv":
        return ops.qgemv(a, w, epilogue=epilogue, residual=s["res"], out_f32=s["f32"])
    return ops.qgemm_grouped(a, w, s["offsets"], epilogue=epilogue, residual=s["res"], out_f32=s["f32"])


def _values(codes, scale):
    """The bf16 values that INT8 codes with one scale per row stand for."""
    out = torch.empty(codes.shape, dtype=torch.bfloat16, device=codes.device)
    return torch.mul(codes, scale[:, None], out=out)


def _sylvester(b):
    """Hadamard matrix of order b divided by sqrt b."""
    i = torch.arange(b, device="cuda")
    v = i[:, None] & i[None, :]
    odd = sum((v >> j) & 1 for j in range(b.bit_length())) & 1
    return (1 - 2 * odd).float() / math.sqrt(b)


def _nibbles(codes, dtype):
    """[.., k/2] bytes -> [.., k] signed values, even k from the low nibble."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return (q ^ 8).to(dtype) - 8


def _finish(y, s):
    if s["epilogue"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif s["epilogue"] == "residual":
        y = y + s["res"].to(y.dtype)
    return y


def _run_plain(s):
    if s["op"] == "norm":
        h = s["x"].float()
        out = {}
        if s["res"] is not None:
            h = h + s["res"].float()
            out["sum"] = h.to(torch.bfloat16)
        y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        if s["w"] is not None:
            y = y * s["w"]
        if s["had"]:
            y = (y.view(-1, s["had"]) @ s["rotation"]).view_as(y)
        out["scale"] = y.abs().amax(1) / 127
        step = torch.where(out["scale"] > 0, out["scale"], 1.0)
        codes = torch.round(y / step[:, None]).clamp(-127, 127).to(torch.int8)
        return dict(out, value=_values(codes, out["scale"]))
    k = s["k"]
    w = _nibbles(s["w4"], torch.float32)
    w = (w.unflatten(-1, (k // GROUP, GROUP)) * s["w4_scale"].mT.unsqueeze(-1)).flatten(-2)
    x = s["codes"].float() * s["scale"][:, None]
    if s["op"] == "gemv":
        y = x @ w.mT
    else:  # the experts' rows side by side, each padded to the longest
        at = s["offsets"][:-1, None] + torch.arange(s["most"], device="cuda")
        y = torch.bmm(x[at.clamp(max=s["rows"] - 1)], w.mT)
        row = torch.arange(s["rows"], device="cuda", dtype=torch.int32)
        e = torch.searchsorted(s["offsets"][1:].contiguous(), row, right=True)
        y = y[e, row - s["offsets"][e]]
    y = _finish(y, s)
    return y if s["f32"] else y.to(torch.bfloat16)


# ---------------------------------------------------------------- 64 bits --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() if s["res"] is None else s["x"].double() + s["res"].double()
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / case["k"] + EPS)
        if s["w"] is not None:
            y = y * s["w"].double()
        if case["had"]:
            b, step = case["had"], 1
            y = y.reshape(case["m"], -1, b)
            while step < b:  # sums and differences of elements `step` apart
                p = y.reshape(case["m"], -1, b // (2 * step), 2, step)
                y = torch.stack((p[..., 0, :] + p[..., 1, :], p[..., 0, :] - p[..., 1, :]), -2)
                step *= 2
            y = y.reshape(case["m"], case["k"]) / math.sqrt(b)
        scale = y.abs().amax(1) / 127
        q = torch.round(y / scale.clamp(min=1e-300)[:, None])
        out = {"value": q * scale[:, None], "scale": scale}
        return dict(out, sum=h) if case["residual"] else out
    k, n = case["k"], case["n"]
    bounds = [0, case["m"]] if case["op"] == "gemv" else s["offsets"].tolist()
    w4, w4_scale = s["w4"].view(-1, n, k // 2), s["w4_scale"].view(-1, k // GROUP, n)
    y = torch.empty((bounds[-1], n), dtype=torch.float64, device="cuda")
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if a == b:
            continue
        w = torch.empty((n, k), dtype=torch.float64, device="cuda")
        w[:, 0::2] = ((w4[e] & 15) ^ 8).double() - 8
        w[:, 1::2] = ((w4[e] >> 4) ^ 8).double() - 8
        w *= w4_scale[e].double().repeat_interleave(GROUP, 0).mT
        y[a:b] = (s["codes"][a:b].double() @ w.mT) * s["scale"][a:b].double()[:, None]
    if case["epilogue"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif case["epilogue"] == "residual":
        y = y + s["res"].double()
    return y
