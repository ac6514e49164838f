"""The mixture-of-experts layer: the router on the normed stream, and calls on two streams and in a captured graph.  The
reference and its bound are those of test_gpu_ffn."""
import pytest
import torch

from test_gpu_ffn import _close, _inputs, _ref, _weight

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ffn():
    from video_dit_mixed_gb300 import ffn as f
    return f


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _experts(ops, g, e, hid, f, b=64):
    return tuple(ops.pack_experts((torch.randn((e,) + s, generator=g) * 0.05).cuda(), b) for s in ((f, hid), (hid, f)))


@pytest.mark.parametrize("t,e,k", [(1, 4, 2), (30, 8, 2), (400, 4, 1)])
def test_normed_router(ffn, ops, t, e, k):
    hid, f, b, eps = 256, 384, 64, 1e-6
    g, x, r, nw = _inputs(t, hid, 7 + t)
    x[t // 2] *= 30                    # (a loud token: its logits differ from the stream's by its norm)
    up, down = _experts(ops, g, e, hid, f, b)
    router = torch.randn((e, hid), generator=g) * 0.3
    layer = ffn.MoEFFN(router.cuda(), up, down, k, nw.cuda(), b, eps, normed_router=True)
    y, h = layer(x.cuda(), r.cuda())
    layer.check()
    hb = h.double().cpu()
    assert torch.equal(h.cpu(), (x.float() + r.float()).to(torch.bfloat16))
    logits = (hb / (hb.square().mean(1, keepdim=True) + eps).sqrt() * nw.double()) @ router.double().mT
    top = logits.topk(k, dim=1)
    probs, full = torch.softmax(top.values, 1), x.double() + r.double()
    ref = torch.zeros((t, hid), dtype=torch.float64)
    for i in range(e):
        tok, slot = (top.indices == i).nonzero(as_tuple=True)
        if len(tok):
            out = _ref(full[tok], nw.double(), _weight(up.i4_codes[i], up.i4_scales[i]),
                       _weight(down.i4_codes[i], down.i4_scales[i]), b)
            ref.index_add_(0, tok, out * probs[tok, slot, None])
    _close(y, ref)


@pytest.mark.parametrize("t", [3, 40, 500])
def test_streams_and_graph(ffn, ops, t):
    hid, f, e, k = 256, 640, 4, 2
    g = torch.Generator().manual_seed(t)
    layers = [ffn.MoEFFN((torch.randn((e, hid), generator=g) * 0.3).cuda(), *_experts(ops, g, e, hid, f), k)
              for _ in range(2)]
    args = [tuple(torch.randn((t, hid), generator=g).to(torch.bfloat16).cuda() for _ in range(2)) for _ in layers]
    want = [[o.clone() for o in layer(*a)] for layer, a in zip(layers, args)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(15):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(layers[i](*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for pair in got[i] for a, b in zip(pair, want[i]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layers[0](*args[0])
    for _ in range(2):
        for o in out:
            o.zero_()
        graph.replay()
        layers[1](*args[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[0]))
    for layer in layers:
        layer.check()
