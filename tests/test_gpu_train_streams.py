"""The embedding and the layer norm with their gradients on several streams at once, and in graphs that share a
memory pool: the bits of a call by itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
# tokens, vocabulary, width: one block, several sorting blocks, rows off 16 bytes, runs over many blocks
SIZES = [(48, 300, 512, BF16), (2500, 5000, 1023, F32), (8191, 9000, 1024, BF16), (5000, 100, 2049, BF16),
         (140000, 900, 64, BF16)]


@pytest.fixture(scope="module")
def dgl():
    from dense_gemm_linear_gb300 import _build
    _build.build()
    import dense_gemm_linear_gb300 as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def inputs():
    g = torch.Generator("cuda").manual_seed(1)

    def some(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    return [(torch.randint(0, V, (T,), device="cuda", generator=g), some(T, d).to(t), some(T, d).to(t), some(d), some(d), V)
            for T, V, d, t in SIZES]


def work(dgl, tokens, x, dy, w, b, V):
    y, mean, rstd = dgl.layer_norm(x, w, b)
    dx, dw, db = dgl.layer_norm_grad(dy, x, mean, rstd, w)
    dW = dgl.embedding_grad(tokens, dx, V, dw_dtype=dgl.OUT_F32)
    more = dgl.embedding_grad(tokens, dy, V, dW=dW.clone(), accumulate=True)
    return y, mean, rstd, dx, dw, db, dW, more, dgl.embedding(tokens, more)


def test_streams_at_once(dgl, inputs):
    want = [work(dgl, *i) for i in inputs]
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for k in range(10):
        for j, s in enumerate(streams):
            n = (k + j) % len(inputs)
            with torch.cuda.stream(s):
                got.append((n, work(dgl, *inputs[n])))
    torch.cuda.synchronize()
    for n, outputs in got:
        assert all(torch.equal(p, q) for p, q in zip(outputs, want[n]))


def test_graphs_of_one_pool(dgl, inputs):
    """Replayed one after the other in the order of their capture, as graphs of one pool may be."""
    want = [work(dgl, *i) for i in inputs]
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for i in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outputs = work(dgl, *i)
        graphs.append((graph, outputs))
    for _ in range(3):
        for _, outputs in graphs:
            for t in outputs:
                t.zero_()
        for graph, _ in graphs:
            graph.replay()
        for (_, outputs), expected in zip(graphs, want):
            assert all(torch.equal(p, q) for p, q in zip(outputs, expected))
