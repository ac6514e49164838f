"""Feed-forward layers on several streams at once and in CUDA graphs: every result equals the one of the call alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ffn():
    from video_dit_mixed_gb300 import ffn as f
    return f


@pytest.fixture(scope="module")
def ops():
    from video_dit_mixed_gb300 import ops as o
    return o


def _dense(ffn, ops, hid, f, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    up, down = (ops.pack_weights(torch.randn(s, generator=g, device="cuda") * 0.02, 64) for s in ((f, hid), (hid, f)))
    return ffn.FFN(up, down, torch.rand(hid, generator=g, device="cuda") + 0.5)


def _tokens(t, hid, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return tuple(torch.randn((t, hid), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))


@pytest.mark.parametrize("t", [20, 600])
def test_two_layers_on_two_streams(ffn, ops, t):
    hid, f = 640, 2560
    layers = [_dense(ffn, ops, hid, f, s) for s in (1, 2)]
    args = [_tokens(t, hid, s) for s in (3, 4)]
    want = [[o.clone() for o in layer(*a)] for layer, a in zip(layers, args)]
    assert not torch.equal(want[0][0], want[1][0])
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(40):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(layers[i](*args[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for y, h in got[i]:
            assert torch.equal(y, want[i][0]) and torch.equal(h, want[i][1])


@pytest.mark.parametrize("t", [20, 300])
def test_a_captured_layer_beside_a_larger_one(ffn, ops, t):
    """The graph keeps no address of a buffer that a later call replaces, and writes into nobody's tensors."""
    small, large = _dense(ffn, ops, 256, 1024, 5), _dense(ffn, ops, 1280, 5120, 6)
    x, r = _tokens(t, 256, 7)
    want = [o.clone() for o in small(x, r)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = small(x, r)
    big = _tokens(t, 1280, 8)
    ref = [o.clone() for o in large(*big)]
    others = [torch.full((1 << 18,), i, dtype=torch.uint8, device="cuda") for i in range(64)]  # (where a freed buffer was)
    for _ in range(3):
        for o in got:
            o.zero_()
        graph.replay()
        y, h = large(*big)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(y, ref[0]) and torch.equal(h, ref[1])
        assert all(bool((o == i).all()) for i, o in enumerate(others))
