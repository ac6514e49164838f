"""The calls around a feed-forward layer's products in device-selected branches of a captured graph, in every form that a
launch may take (one kernel or several, clusters, launches that start early)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _norm(ops, g, m):
    k = 640
    x, r = (torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    w, gate = torch.rand(k, generator=g, device="cuda"), torch.randn((2, k), generator=g, device="cuda")
    seg = torch.randint(0, 2, (m,), generator=g, device="cuda", dtype=torch.int32)
    out = ops.int8_act(torch.zeros((m, k), dtype=torch.int8, device="cuda"), torch.zeros(m, device="cuda"))
    h = torch.zeros_like(x)
    return [out.i8_codes, out.row_scale, h], lambda: ops.gated_rmsnorm_quant(x, r, w, w, gate, segment=seg, had_block=64,
                                                                            out=out, sum_out=h)


def _route(ops, g, t):
    e = 64
    z, b = torch.randn((t, e), generator=g, device="cuda"), torch.randn(e, generator=g, device="cuda") * 0.1
    out = ops.moe_route(z, 4, ops.SCORE_SIGMOID, bias=b)
    ws = torch.empty(max(1, ops.moe_route_workspace_bytes(t, e)), dtype=torch.uint8, device="cuda")
    return list(out), lambda: ops.moe_route(z, 4, ops.SCORE_SIGMOID, bias=b, out=out, ws=ws)


def _combine(ops, g, t):
    d, w = torch.randn((2 * t, 256), generator=g, device="cuda"), torch.rand((t, 2), generator=g, device="cuda")
    rows = torch.randint(0, 2 * t, (t, 2), generator=g, device="cuda", dtype=torch.int32)
    y = torch.zeros((t, 256), dtype=torch.bfloat16, device="cuda")
    return [y], lambda: ops.moe_combine(d, rows, w, out=y)


def _lowrank(ops, g, m):
    n, k, r = 320, 640, 32
    a = (torch.randn((3, r, k), generator=g, device="cuda") * k ** -0.5).to(torch.bfloat16)
    w = ops.LowRank(a, torch.randn((3, n, r), generator=g, device="cuda").to(torch.bfloat16))
    ids = torch.randint(-1, 3, (m,), generator=g, device="cuda", dtype=torch.int32)
    x, base = torch.randn((m, k), generator=g, device="cuda").to(torch.bfloat16), torch.randn((m, n), generator=g, device="cuda")
    y = torch.zeros((m, n), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(1, ops.lowrank_workspace_bytes(m, r)), dtype=torch.uint8, device="cuda")
    return [y], lambda: ops.lowrank_add(x, w, ids, base, ops.EPI_GELU, out=y, ws=ws)


CASES = [(f, m) for f, sizes in ((_norm, (5, 900)), (_route, (3, 700)), (_combine, (4, 700)), (_lowrank, (1, 20, 300, 5000)))
         for m in sizes]


@pytest.mark.parametrize("make,m", CASES)
def test_branch(ops, make, m):
    outs, call = make(ops, torch.Generator(device="cuda").manual_seed(m), m)
    call()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    stream, body = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        sw = ops.GraphSwitch(stream, body, word, ops.MODE_INT8, 1)
        with sw.branch(0):
            call()
        sw.close()
    for mode in (ops.MODE_INT8, ops.MODE_BF16, ops.MODE_INT8):
        word.fill_(mode)
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w) if mode == ops.MODE_INT8 else not o.any()


def test_outputs_of_another_size_are_refused(ops):
    z = torch.zeros((4, 8), device="cuda")
    r = ops.moe_route(z, 2)
    assert ops.moe_route(z, 2, out=r) is r
    for bad in (lambda: ops.moe_route(z[:3], 2, out=r), lambda: ops.moe_route(z, 3, out=r),
                lambda: ops.moe_route(torch.zeros((4, 9), device="cuda"), 2, out=r),
                lambda: ops.moe_route(torch.zeros((40, 8), device="cuda"), 2, ws=torch.zeros(8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
