"""AdamW on several streams at once, and in graphs that share a memory pool: the bits of a step by itself."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# one launch of few tensors, more than a small table holds, more than one launch does, one large
SIZES = [[900, 33], [100 + i for i in range(60)], [(7 * i) % 50 + 1 for i in range(700)], [3_000_001]]


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


def make(dgl, n, bits):
    gen = torch.Generator(device="cuda").manual_seed(n)
    params = [torch.randn(k, device="cuda", generator=gen) for k in SIZES[n]]
    params = [p.to(BF16) if i % 2 else p for i, p in enumerate(params)]
    grads = [torch.randn(k, device="cuda", generator=gen).to(F32 if i % 3 else BF16) for i, k in enumerate(SIZES[n])]
    return dgl.AdamW(params, grads, master=True, state_bits=bits, seed=n)


def outputs(opt):
    scales = [] if opt.state_bits == 32 else [*opt.exp_avg_scale, *opt.exp_avg_sq_scale]
    masters = [m for m in opt.master if m is not None]
    return [t.view(torch.uint8) for t in (*opt.params, *masters, *opt.exp_avg, *opt.exp_avg_sq, *scales, opt.steps)]


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(outputs(a), outputs(b)))


@pytest.mark.parametrize("bits", [8, 32])
def test_streams_at_once(dgl, bits):
    """Optimizers of their own on four streams, their steps enqueued in turn."""
    alone, together = ([make(dgl, n, bits) for n in range(len(SIZES))] for _ in range(2))
    for opt in alone:
        for _ in range(6):
            opt.step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in SIZES]
    for k in range(6):
        for opt, s in zip(together, streams):
            if k % 2:
                opt.step(stream=s)
            else:
                with torch.cuda.stream(s):
                    opt.step()
    torch.cuda.synchronize()
    assert all(equal(a, b) for a, b in zip(alone, together))


@pytest.mark.parametrize("bits", [8, 32])
def test_graphs_of_one_pool(dgl, bits):
    """Captured with a gradient's arithmetic whose memory the pool hands out again, replayed in the order of capture."""
    alone, together = ([make(dgl, n, bits) for n in range(len(SIZES))] for _ in range(2))
    lr = torch.full((1,), 1e-3, device="cuda")

    def step(opt):
        opt.step([0.5 * g for g in opt.grads], lr=lr, grad_scale=2.0 * lr / lr)

    for _ in range(4):
        for opt in alone:
            step(opt)
    pool, graphs = torch.cuda.graph_pool_handle(), []
    for opt in together:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            step(opt)
        graphs.append(graph)
    for _ in range(4):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(equal(a, b) for a, b in zip(alone, together))


def test_two_optimizers_of_one_model(dgl):
    """Halves of a model's tensors in two optimizers, on two streams at once, give what one for all gives in 32 bits."""
    whole, parts = make(dgl, 1, 32), make(dgl, 1, 32)
    n = len(SIZES[1]) // 2
    halves = [dgl.AdamW(parts.params[a:b], parts.grads[a:b], master=parts.master[a:b]) for a, b in ((0, n), (n, None))]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in halves]
    for _ in range(3):
        whole.step()
        for opt, s in zip(halves, streams):
            opt.step(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(whole.params, parts.params))
