"""Performance cases of the operators around a routed, adapted and modulated feed-forward layer.

Four operators that a quantized feed-forward layer of a large model runs next to
its norm, quantization and products, from a single token to a whole video:

``norm``     RMS norms before and after a block: the branch's norm, its gate and the
             scaled residual, the next norm with scale and shift, then a rotation and
             per-token INT8 codes, or bf16
``route``    routing to experts: softmax or sigmoid scores, a bias for balance, groups
             of experts, top-k, renormalised weights, and the rows sorted by expert
``combine``  the weighted sum of each token's rows of expert outputs
``lowrank``  low-rank adapters of many requests beside a shared projection

``listed()`` gives the named cases, ``draw(rng)`` more of the same ranges.
``prepare`` makes a case's inputs, ``run`` one pass: in plain torch operations
when ``own`` is false, through the library when it is true.  ``exact`` is the
operators' definition in 64 bits.  Sums and statistics are in 32 bits or more;
scores are compared in 64; 8-bit results are returned as the values they stand for.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6
MAX_TOKENS = 17776  # 13 x 30 x 45 latent positions and 226 text tokens
TEXT = 226
MAX_NORM = MAX_TOKENS * 1920  # elements of the largest norm
MAX_SCORES = MAX_TOKENS * 64  # logits of the largest routing
MAX_ROWS = 2 * MAX_TOKENS * 1920  # expert output elements of the largest sum
MAX_ADAPTED = MAX_TOKENS * 7680  # outputs of the largest adapted projection
MAX_RANKS = 1024  # ranks over all adapters


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One token of an autoregressive step between two blocks of the 2B-shaped model: latency.
        dict(name="norm_1tok", op="norm", m=1, k=1920, had=64, residual=True, post=True, mod="all", segments=1,
             int8=True),
        # A block boundary of the 2B-shaped model: text and video tokens with a modulation each.
        dict(name="norm_video", op="norm", m=17776, k=1920, had=64, residual=True, post=True, mod="all", segments=2,
             int8=True),
        # An odd number of wide rows, gated only, bf16 for a layer that is not quantized.
        dict(name="norm_wide_odd", op="norm", m=1003, k=7680, had=0, residual=True, post=False, mod="gate",
             segments=3, int8=False),
        # One token to two of eight experts: latency.
        dict(name="route_1tok", op="route", t=1, e=8, k=2, score="softmax", bias=False, groups=1, top_groups=1,
             best=1, renorm=True, bf16=False, dead=0),
        # A prompt's text tokens over many experts in groups, sigmoid scores with a balance bias.
        dict(name="route_text_groups", op="route", t=TEXT, e=256, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, best=2, renorm=True, bf16=False, dead=0),
        # Every video token to two of 64 experts, logits of a bf16 router (many ties).
        dict(name="route_video", op="route", t=17776, e=64, k=2, score="softmax", bias=False, groups=1, top_groups=1,
             best=1, renorm=True, bf16=True, dead=0),
        # Eight single tokens, two experts each.
        dict(name="combine_8tok", op="combine", t=8, k=2, h=1920, f32=True, route=1),
        # Every video token, two experts each, the down projections' float sums.
        dict(name="combine_video", op="combine", t=17776, k=2, h=1920, f32=True, route=2),
        # One token of one request beside the up projection.
        dict(name="lowrank_1tok_up", op="lowrank", m=1, k=1920, n=7680, rank=16, adapters=8, ids="mixed", route=3,
             base="f32", epilogue="gelu", out_f32=False, int8=True),
        # 32 requests a token each, most with an adapter of their own, beside the down projection.
        dict(name="lowrank_32tok_down", op="lowrank", m=32, k=7680, n=1920, rank=16, adapters=64, ids="mixed",
             route=4, base="f32", epilogue="none", out_f32=False, int8=True),
        # An odd number of bf16 rows of a few requests, odd outputs, float result.
        dict(name="lowrank_odd", op="lowrank", m=1003, k=640, n=1111, rank=48, adapters=5, ids="runs", route=5,
             base="bf16", epilogue="residual", out_f32=True, int8=False),
        # The tokens of three videos' requests beside the up projection.
        dict(name="lowrank_video_up", op="lowrank", m=17776, k=1920, n=7680, rank=64, adapters=4, ids="runs",
             route=6, base="bf16", epilogue="gelu", out_f32=False, int8=True),
    ]


def _log(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "route", "combine", "lowrank"])
    if op == "norm":
        k = 128 * _log(rng, 1, 96)
        m = _log(rng, 1, min(MAX_TOKENS, MAX_NORM // k))
        int8 = rng.random() < 0.7
        had = rng.choice([0, 16, 64] + ([256] if k % 256 == 0 else [])) if int8 else 0
        return dict(op=op, m=m, k=k, had=had, residual=rng.random() < 0.8, post=rng.random() < 0.6,
                    mod=rng.choice(["none", "gate", "all", "all"]), segments=min(m, rng.randint(1, 6)), int8=int8)
    if op == "route":
        g = rng.choice([1, 1, 2, 4, 8])
        e = g * _log(rng, 2, 256 // g)
        top = rng.randint(1, g)
        k = rng.randint(1, min(8, e // g * top))
        return dict(op=op, t=_log(rng, 1, min(MAX_TOKENS, MAX_SCORES // e)), e=e, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=g, top_groups=top,
                    best=rng.randint(1, 2), renorm=rng.random() < 0.7, bf16=rng.random() < 0.4,
                    dead=rng.choice([0, 0, 1]))
    if op == "combine":
        k, h = rng.randint(1, 8), 128 * _log(rng, 1, 60)
        return dict(op=op, t=_log(rng, 1, min(MAX_TOKENS, MAX_ROWS // (k * h))), k=k, h=h, f32=rng.random() < 0.6,
                    route=rng.randint(0, 9999))
    k, n = 128 * _log(rng, 1, 60), _log(rng, 16, 7680)
    rank = rng.choice([16, 32, 48, 64])
    return dict(op=op, m=_log(rng, 1, min(MAX_TOKENS, MAX_ADAPTED // max(n, k))), k=k, n=n, rank=rank,
                adapters=_log(rng, 1, MAX_RANKS // rank), ids=rng.choice(["mixed", "runs"]), route=rng.randint(0, 9999),
                base=rng.choice(["f32", "bf16", "none"]), epilogue=rng.choice(["none", "gelu", "residual"]),
                out_f32=rng.random() < 0.3, int8=rng.random() < 0.7)


def _ids(case):
    """The adapter of each row: a request's run of rows, or a row's own; about one row in eight has none (-1)."""
    rng = random.Random(case["route"])
    m, count = case["m"], case["adapters"]

    def one():
        return rng.randrange(count) if rng.random() < 0.875 else -1

    if case["ids"] == "mixed":
        return [one() for _ in range(m)]
    cuts = sorted(rng.randrange(m + 1) for _ in range(rng.randint(1, 7)))
    return [i for a, b in zip([0] + cuts, cuts + [m]) for i in [one()] * (b - a)]


def work(case):
    if case["op"] == "norm":
        m, k, s = case["m"], case["k"], case["segments"]
        words = m * k * (2 + (2 if case["residual"] else 0) + 2 + (1 if case["int8"] else 2))
        words += (4 * m if case["int8"] else 0) + (4 * m if s > 1 and case["mod"] != "none" else 0)
        words += 4 * k * (1 + (1 if case["post"] else 0) + s * {"none": 0, "gate": 1, "all": 3}[case["mod"]])
        return {"bytes": words, "flops": m * k * (12 + (int(math.log2(case["had"])) if case["had"] else 0))}
    if case["op"] == "route":
        t, e, k = case["t"], case["e"], case["k"]
        return {"bytes": t * e * (2 if case["bf16"] else 4) + 16 * t * k + 4 * (e + 1) + (4 * e if case["bias"] else 0),
                "flops": t * e * (4 + k)}
    if case["op"] == "combine":
        t, k, h = case["t"], case["k"], case["h"]
        return {"bytes": t * k * (h * (4 if case["f32"] else 2) + 8) + 2 * t * h, "flops": 2 * t * k * h}
    m, k, n, r = case["m"], case["k"], case["n"], case["rank"]
    live = [i for i in _ids(case) if i >= 0]
    words = len(set(live)) * (2 * r * (k + n) + 4) + len(live) * (k + 4 if case["int8"] else 2 * k) + 4 * m
    words += m * n * ({"f32": 4, "bf16": 2, "none": 0}[case["base"]] + (4 if case["out_f32"] else 2)
                      + (2 if case["epilogue"] == "residual" else 0))
    return {"bytes": words, "flops": 2 * len(live) * r * (k + n)}


# ------------------------------------------------------------------ inputs --

def _activations(g, m, k):
    """bf16 Laplace rows with 0.5 % outlier channels, as a transformer block's branch has them."""
    u = torch.rand((m, k), generator=g, device="cuda") - 0.5
    x = -torch.sign(u) * torch.log1p(-2.0 * u.abs().clamp(max=0.4999999))
    loud = torch.rand((k,), generator=g, device="cuda") < 0.005
    return torch.where(loud, x * 8.0, x).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] == "norm":
        m, k, seg = case["m"], case["k"], case["segments"]
        s["x"] = _activations(g, m, k)
        s["res"] = randn(m, k).to(torch.bfloat16) if case["residual"] else None
        s["w"] = torch.rand((k,), generator=g, device="cuda") + 0.5
        s["post_w"] = torch.rand((k,), generator=g, device="cuda") + 0.5 if case["post"] else None
        s["gate"] = randn(seg, k) * 0.5 if case["mod"] != "none" else None
        s["mod_scale"], s["shift"] = (randn(seg, k) * 0.3, randn(seg, k) * 0.3) if case["mod"] == "all" else (None, None)
        s["res_scale"] = 1.0 if m % 2 else 0.75
        # the first tokens are the text, the others the frames' in runs
        row = torch.arange(m, device="cuda")
        run = torch.where(row < TEXT, 0, 1 + (row - TEXT) * (seg - 1) // max(1, m - TEXT)).clamp(max=seg - 1)
        s["segment"] = run.to(torch.int32) if seg > 1 and case["mod"] != "none" else None
        s["rotation"] = _sylvester(case["had"]) if case["had"] else None  # a constant that a program keeps
        return s
    if case["op"] == "route":
        t, e = case["t"], case["e"]
        s["logits"] = randn(t, e) * 1.5 + randn(e) * 0.5
        if case["dead"] and e // case["groups"] > 1 and case["k"] < e:  # an expert out of service
            s["logits"][:, e // 2] = -math.inf
        if case["bf16"]:
            s["logits"] = s["logits"].to(torch.bfloat16)
        s["balance"] = randn(e) * 0.05 if case["bias"] else None
        s["factor"] = 1.0 if case["renorm"] and case["score"] == "softmax" else 2.5
        return s
    if case["op"] == "combine":
        t, k, h = case["t"], case["k"], case["h"]
        s["d"] = randn(t * k, h) if case["f32"] else randn(t * k, h).to(torch.bfloat16)
        s["w"] = torch.softmax(randn(t, k), 1)
        place = torch.rand((t * k,), generator=g, device="cuda")  # the rows lie by expert, a token's far apart
        s["rows"] = place.argsort().view(t, k).to(torch.int32)
        return s
    m, k, n, r, count = case["m"], case["k"], case["n"], case["rank"], case["adapters"]
    if case["int8"]:
        x = randn(m, k)
        s["codes"] = (x * (127.0 / x.abs().amax(1, keepdim=True))).round_().to(torch.int8)
        s["scale"] = torch.exp(torch.randn((m,), generator=g, device="cuda") * 0.3) * 0.03
    else:
        s["x"] = randn(m, k).to(torch.bfloat16)
    s["a"] = (randn(count, r, k) * k ** -0.5).to(torch.bfloat16)
    s["b"] = (randn(count, n, r) * (0.5 * r ** -0.5)).to(torch.bfloat16)
    s["alpha"] = torch.rand((count,), generator=g, device="cuda") + 0.5
    s["adapter"] = torch.tensor(_ids(case), dtype=torch.int32, device="cuda")
    s["y0"] = None if case["base"] == "none" else randn(m, n).to(torch.float32 if case["base"] == "f32" else torch.bfloat16)
    s["res"] = randn(m, n).to(torch.bfloat16) if case["epilogue"] == "residual" else None
    return s


# ------------------------------------------------------------------ a pass --

def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    from video_dit_mixed_gb300 import ops

    if s["op"] == "norm":
        a, h = ops.gated_rmsnorm_quant(s["x"], s["res"], s["w"], post_weight=s["post_w"], gate=s["gate"],
                                       scale=s["mod_scale"], shift=s["shift"], segment=s["segment"],
                                       residual_scale=s["res_scale"], eps=EPS, had_block=s["had"], quantize=s["int8"])
        if not s["int8"]:
            return {"value": a, "sum": h}
        return {"value": _values(a.i8_codes, a.row_scale), "scale": a.row_scale, "sum": h}
    if s["op"] == "route":
        score = ops.SCORE_SOFTMAX if s["score"] == "softmax" else ops.SCORE_SIGMOID
        return tuple(ops.moe_route(s["logits"], s["k"], score, bias=s["balance"], groups=s["groups"],
                                   top_groups=s["top_groups"], group_best=s["best"], renormalize=s["renorm"],
                                   scale=s["factor"]))
    if s["op"] == "combine":
        return ops.moe_combine(s["d"], s["rows"], s["w"])
    x = ops.int8_act(s["codes"], s["scale"]) if s["int8"] else s["x"]
    epilogue = {"none": ops.EPI_NONE, "gelu": ops.EPI_GELU, "residual": ops.EPI_RESIDUAL}[s["epilogue"]]
    return ops.lowrank_add(x, ops.LowRank(s["a"], s["b"], s["alpha"]), s["adapter"], s["y0"], epilogue=epilogue,
                           residual=s["res"], out_f32=s["out_f32"])


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


def _plain_norm(s):
    def normed(v, w):
        return v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * w

    def of_row(v):
        return v if s["segment"] is None else v[s["segment"]]

    h = s["x"].float()
    if s["post_w"] is not None:
        h = normed(h, s["post_w"])
    if s["gate"] is not None:
        h = h * of_row(s["gate"])
    if s["res"] is not None:
        h = h + s["res"].float() * s["res_scale"]
    y = normed(h, s["w"])
    if s["shift"] is not None:
        y = y * (1 + of_row(s["mod_scale"])) + of_row(s["shift"])
    out = {"sum": h.to(torch.bfloat16)}
    if not s["int8"]:
        return dict(out, value=y.to(torch.bfloat16))
    if s["had"]:
        y = (y.view(-1, s["had"]) @ s["rotation"]).view_as(y)
    out["scale"] = y.abs().amax(1) / 127
    step = torch.where(out["scale"] > 0, out["scale"], 1.0)
    codes = torch.round(y / step[:, None]).clamp(-127, 127).to(torch.int8)
    return dict(out, value=_values(codes, out["scale"]))


def _plain_route(s):
    t, e = s["logits"].shape
    k, g = s["k"], s["groups"]
    logits = s["logits"].double()
    if s["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-logits))
    key = p if s["balance"] is None else p + s["balance"].double()
    order = logits if s["balance"] is None else key  # both scores rise with the logit
    if g > 1:
        best = key.view(t, g, e // g).sort(dim=2, descending=True).values[:, :, :min(s["best"], e // g)].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        allowed = torch.zeros((t, g), dtype=torch.bool, device=key.device).scatter(1, kept, True)
        # (an expert of a kept group comes before every other, however low its logit)
        outside = ~allowed.repeat_interleave(e // g, 1)
        first = order.sort(dim=1, descending=True, stable=True).indices
        first = first.gather(1, outside.gather(1, first).to(torch.int8).sort(dim=1, stable=True).indices)
    else:
        first = order.sort(dim=1, descending=True, stable=True).indices
    experts = first[:, :k].contiguous()
    w = p.gather(1, experts)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    w = (w * s["factor"]).float()
    by_expert, place = experts.flatten().sort(stable=True)
    rows = torch.empty_like(place)
    rows[place] = torch.arange(t * k, device=place.device)
    offsets = torch.searchsorted(by_expert, torch.arange(e + 1, device=place.device))
    return experts.int(), w, rows.view(t, k).int(), (place // k).int(), offsets.int()


def _plain_combine(s):
    return (s["d"][s["rows"]].float() * s["w"].unsqueeze(-1)).sum(1).to(torch.bfloat16)


def _plain_lowrank(s):
    count, r, k = s["a"].shape
    m, n = len(s["adapter"]), s["b"].shape[1]
    x = s["codes"].float() * s["scale"][:, None] if s["int8"] else s["x"].float()
    chosen = s["adapter"][:, None] == torch.arange(count, device=x.device)  # [m, count]; -1 has none
    v = (x @ s["a"].float().view(count * r, k).mT).view(m, count, r)
    v = torch.where(chosen[:, :, None], v * s["alpha"][:, None], 0.0)
    y = v.view(m, count * r) @ s["b"].float().mT.reshape(count * r, n)
    if s["y0"] is not None:
        y = y + s["y0"].float()
    if s["epilogue"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif s["epilogue"] == "residual":
        y = y + s["res"].float()
    return y if s["out_f32"] else y.to(torch.bfloat16)


_PLAIN = {"norm": _plain_norm, "route": _plain_route, "combine": _plain_combine, "lowrank": _plain_lowrank}


# ---------------------------------------------------------------- 64 bits --

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _exact_norm(case, s):
    m, k = case["m"], case["k"]
    at = torch.zeros(m, dtype=torch.long, device="cuda") if s["segment"] is None else s["segment"].long()
    u = s["x"].double()
    if case["post"]:
        u = u / torch.sqrt(u.square().sum(1, keepdim=True) / k + EPS) * s["post_w"].double()
    h = u if s["gate"] is None else u * s["gate"].double()[at]
    if case["residual"]:
        h = h + s["res_scale"] * s["res"].double()
    y = h / torch.sqrt(h.square().sum(1, keepdim=True) / k + EPS) * s["w"].double()
    if case["mod"] == "all":
        y = y + y * s["mod_scale"].double()[at] + s["shift"].double()[at]
    if not case["int8"]:
        return {"sum": h, "value": y}
    if case["had"]:
        b, step = case["had"], 1
        y = y.reshape(m, -1, b)
        while step < b:  # sums and differences of elements `step` apart
            p = y.reshape(m, -1, b // (2 * step), 2, step)
            y = torch.stack((p[..., 0, :] + p[..., 1, :], p[..., 0, :] - p[..., 1, :]), -2)
            step *= 2
        y = y.reshape(m, k) / math.sqrt(b)
    scale = y.abs().amax(1) / 127
    q = torch.round(y / scale.clamp(min=1e-300)[:, None])
    return {"value": q * scale[:, None], "scale": scale, "sum": h}


def _exact_route(case, s):
    t, e, k, g = case["t"], case["e"], case["k"], case["groups"]
    z = s["logits"].double()
    p = torch.softmax(z, 1) if case["score"] == "softmax" else torch.sigmoid(z)
    key = p + s["balance"].double() if case["bias"] else p
    number = torch.arange(e, device="cuda").expand(t, e)

    def first_largest(v, left):
        """The lowest place of the largest value among those left."""
        top = torch.where(left, v, -math.inf).amax(1, keepdim=True)
        return torch.where(left & (v == top), number[:, :v.shape[1]], e).amin(1, keepdim=True)

    left = torch.ones((t, e), dtype=torch.bool, device="cuda")
    if g > 1:
        size = e // g
        groups = torch.stack([key[:, i * size:(i + 1) * size].topk(min(case["best"], size), 1).values.sum(1)
                              for i in range(g)], 1)
        open_, kept = torch.ones((t, g), dtype=torch.bool, device="cuda"), torch.zeros((t, g), dtype=torch.bool, device="cuda")
        for _ in range(case["top_groups"]):
            i = first_largest(groups, open_)
            open_.scatter_(1, i, False)
            kept.scatter_(1, i, True)
        left = kept.repeat_interleave(size, 1)
    order = key if case["bias"] else z
    experts = []
    for _ in range(k):
        i = first_largest(order, left)
        left = left.scatter(1, i, False)
        experts.append(i)
    experts = torch.cat(experts, 1)
    w = p.gather(1, experts)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    flat = experts.flatten()
    counts = torch.bincount(flat, minlength=e)
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    token = torch.cat([(flat == i).nonzero().flatten() for i in range(e)])
    rows = torch.empty_like(flat)
    rows[token] = torch.arange(t * k, device="cuda")
    return experts, w * s["factor"], rows.view(t, k), token // k, offsets


def _exact_combine(case, s):
    y = torch.zeros((case["t"], case["h"]), dtype=torch.float64, device="cuda")
    for j in range(case["k"]):
        y += s["d"][s["rows"][:, j].long()].double() * s["w"][:, j, None].double()
    return y


def _exact_lowrank(case, s):
    x = s["codes"].double() * s["scale"].double()[:, None] if case["int8"] else s["x"].double()
    y = torch.zeros((case["m"], case["n"]), dtype=torch.float64, device="cuda")
    if s["y0"] is not None:
        y += s["y0"].double()
    for i in range(case["adapters"]):
        at = (s["adapter"] == i).nonzero().flatten()
        if len(at):
            y[at] += (x[at] @ s["a"][i].double().mT) @ s["b"][i].double().mT * s["alpha"][i].double()
    if case["epilogue"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif case["epilogue"] == "residual":
        y = y + s["res"].double()
    return y


_EXACT = {"norm": _exact_norm, "route": _exact_route, "combine": _exact_combine, "lowrank": _exact_lowrank}
