"""Products that pass no workspace: on several streams at once, in graphs replayed after other
calls have outgrown the buffers, and beside one another.  Every result must be bit for bit that
of the call alone (the kernels' sums have a fixed order)."""
import pytest

import bit_weight_only_w4_b200 as w4
from tests.gpu_util import skip_without_gpu, torch_mod
from tests.test_gpu_epilogue import Layer

pytestmark = pytest.mark.gpu


def product(L, X, **kw):
    return w4.w4a16_gemm_epi(X, L.qw, L.sc, L.zr, L.group, activation="silu", **kw)


def plain(L, X, **kw):
    return w4.w4a16_gemm(X, L.qw, L.sc, L.zr, L.group, **kw)


@pytest.mark.parametrize("call", [product, plain])
@pytest.mark.parametrize("warm", [False, True])
def test_graph_outlives_the_buffers_of_other_calls(call, warm):
    skip_without_gpu()
    torch = torch_mod()
    small, large = Layer(1, 1024, 2048, 128), Layer(2, 2048, 8192, 128)
    X, big = small.acts(4), large.acts(64)
    want, want_big = call(small, X), call(large, big)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    if warm:
        call(small, X, stream=s)
    Y = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(small, X, Y=Y)
        call(small, X, Y=Y)
    assert torch.equal(call(large, big), want_big)    # more rows and channels: larger buffers,
    torch.cuda.synchronize()
    assert torch.equal(call(large, big, stream=s, Y=torch.empty_like(want_big)), want_big)   # ... also on the graph's stream
    torch.cuda.synchronize()
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in [1 << 20, 8 << 20, 12 << 20, 20 << 20] * 6]
    for _ in range(3):
        Y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, want)
    assert all(bool((t == 255).all()) for t in junk)
    assert torch.equal(call(small, X), want)
    w4.w4_check_device_error()


def test_graphs_replayed_beside_each_other_and_eager_calls():
    skip_without_gpu()
    torch = torch_mod()
    L = Layer(3, 2048, 4096, 128)
    Xs = [L.acts(6) for _ in range(3)]
    want = [product(L, X) for X in Xs]
    streams = [torch.cuda.Stream() for _ in Xs]
    graphs, Ys = [], []
    for X, y in zip(Xs[:2], want):
        g, Y = torch.cuda.CUDAGraph(), torch.zeros_like(y)
        with torch.cuda.graph(g):
            for _ in range(20):
                product(L, X, Y=Y)
        graphs.append(g)
        Ys.append(Y)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [product(L, Xs[2]) for _ in range(20)]
        torch.cuda.synchronize()
        assert torch.equal(Ys[0], want[0]) and torch.equal(Ys[1], want[1])
        assert all(torch.equal(y, want[2]) for y in eager)
    w4.w4_check_device_error()


@pytest.mark.parametrize("M", [1, 20, 100])
def test_unordered_streams(M):
    skip_without_gpu()
    torch = torch_mod()
    layers = [Layer(4, 1024, 4096, 128), Layer(5, 2048, 2048, 64)]
    Xs = [L.acts(M) for L in layers]
    s_inv = [torch.rand(L.K, device="cuda") + 0.5 for L in layers]
    want = [product(L, X, s_inv=f) for L, X, f in zip(layers, Xs, s_inv)]
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, product(layers[i], Xs[i], s_inv=s_inv[i])))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i, y in got)
    w4.w4_check_device_error()
