"""Embedding lookup and its gradient against their definitions in fp64.

u is fp32's unit roundoff: a row of dW that n tokens add to takes at most n + 8
roundings of fp32, each at most u of the sum of magnitudes; a bf16 dW half a
step more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0**-24
IGNORE = -100


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


def half_step(t):
    return torch.finfo(t).eps / 2


def make_tokens(T, V, kind, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    u = torch.rand(T, device="cuda", generator=gen)
    if kind == "one":  # all the same
        t = torch.full((T,), V - 1, dtype=torch.int64, device="cuda")
    elif kind == "all":  # as many different ones as there are
        t = torch.arange(T, device="cuda").flip(0) % V
    elif kind == "ignored":
        return torch.full((T,), IGNORE, dtype=torch.int64, device="cuda")
    else:  # a few frequent ones, many rare ones
        t = (torch.exp(u * torch.log(torch.tensor(float(V)))) - 1).long().clamp(0, V - 1)
    if kind == "mixed":
        t = torch.where(torch.rand(T, device="cuda", generator=gen) < 0.1, IGNORE, t)
        if T > 20:
            t[3], t[11], t[17] = V, -1, V + 2**40
    return t


def grad64(tokens, dY, V, scale, dW=None):
    keep = ((tokens != IGNORE) & (tokens >= 0) & (tokens < V)).nonzero()[:, 0]
    terms = dY[keep].double() * scale
    start = torch.zeros(V, dY.shape[1], dtype=torch.float64, device="cuda") if dW is None else dW.double()
    sums = start.index_put((tokens[keep],), terms, accumulate=True)
    sizes = start.abs().index_put((tokens[keep],), terms.abs(), accumulate=True)
    count = torch.bincount(tokens[keep], minlength=V).double()[:, None]
    return sums, sizes, count


@pytest.mark.parametrize("w_dtype,y_dtype", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
@pytest.mark.parametrize("T,V,d", [(1, 1, 1), (5, 9, 3), (40, 100, 64), (333, 4095, 130), (1000, 50, 1025),
                                   (77, 31, 4096)])
def test_lookup(dgl, T, V, d, w_dtype, y_dtype):
    gen = torch.Generator(device="cuda").manual_seed(1)
    W = torch.randn(V, d, device="cuda", generator=gen).to(w_dtype)
    tokens = make_tokens(T, V, "mixed")
    code = dgl.OUT_BF16 if y_dtype == BF16 else dgl.OUT_F32
    for scale in (1.0, 22.627):
        Y = dgl.embedding(tokens, W, scale=scale, out_dtype=code)
        real = (tokens != IGNORE) & (tokens >= 0) & (tokens < V)
        at = torch.where(real, tokens, 0)
        # one product in fp32, rounded once to nearest even
        want = torch.where(real[:, None], W[at].float() * torch.tensor(scale, device="cuda"), 0.0).to(y_dtype)
        want[~real & (tokens != IGNORE)] = float("nan")
        assert torch.equal(Y.isnan(), want.isnan())
        assert torch.equal(Y.nan_to_num(), want.nan_to_num())


GRADS = [(1, 1, 1, "all"), (1, 300, 64, "all"), (2, 7, 5, "one"), (31, 4095, 512, "mixed"), (48, 50, 130, "zipf"),
         (700, 1000, 1024, "mixed"), (2048, 513, 96, "zipf"), (2049, 512, 72, "mixed"), (3000, 100000, 40, "all"),
         (5000, 77, 264, "one"), (9000, 50257, 128, "mixed"), (16384, 511, 24, "all"), (16385, 140000, 17, "zipf"),
         (40000, 3, 33, "zipf"), (70001, 262145, 8, "mixed"), (131072, 1024, 16, "zipf"), (4096, 600, 2056, "mixed"),
         (600, 90, 8200, "zipf"), (200, 64, 64, "ignored")]


@pytest.mark.parametrize("y_dtype,dw_dtype,add", [(BF16, BF16, False), (BF16, F32, False), (BF16, F32, True),
                                                  (F32, F32, False), (F32, BF16, False), (F32, F32, True)])
@pytest.mark.parametrize("T,V,d,kind", GRADS)
def test_gradient(dgl, T, V, d, kind, y_dtype, dw_dtype, add):
    gen = torch.Generator(device="cuda").manual_seed(2)
    tokens = make_tokens(T, V, kind)
    dY = torch.randn(T, d, device="cuda", generator=gen).to(y_dtype)
    dY[tokens == IGNORE] = float("nan")  # padding's rows are not read into anything
    scale = 0.75
    dW = torch.randn(V, d, device="cuda", generator=gen) if add else torch.full((V, d), float("nan"), device="cuda").to(dw_dtype)
    sums, sizes, count = grad64(tokens, dY, V, scale, dW if add else None)
    before = dW.clone()
    got = dgl.embedding_grad(tokens, dY, V, scale=scale, dW=dW, accumulate=add)
    assert got is dW
    tol = half_step(dw_dtype) * sums.abs() * (dw_dtype == BF16) + (count + 8) * U * sizes
    bad = ~((got.double() - sums).abs() <= tol)
    assert not bad.any(), f"{int(bad.sum())} off, first {bad.nonzero()[0].tolist()}"
    unreached = count[:, 0] == 0
    if add:
        assert torch.equal(got[unreached], before[unreached])
    else:
        assert not got[unreached].any()
    if not add:
        code = dgl.OUT_BF16 if dw_dtype == BF16 else dgl.OUT_F32
        assert torch.equal(dgl.embedding_grad(tokens, dY, V, scale=scale, dw_dtype=code), got)


@pytest.mark.parametrize("dw_dtype,add", [(BF16, False), (F32, False), (F32, True)])
def test_more_tokens_than_are_sorted_at_once(dgl, dw_dtype, add):
    T, V, d = 131072 * 2 + 777, 5000, 16
    tokens = make_tokens(T, V, "mixed")
    gen = torch.Generator(device="cuda").manual_seed(2)
    dY = torch.randn(T, d, device="cuda", generator=gen).bfloat16()
    dW = torch.randn(V, d, device="cuda", generator=gen).to(dw_dtype)
    sums, sizes, count = grad64(tokens, dY, V, 1.0, dW if add else None)
    dgl.embedding_grad(tokens, dY, V, dW=dW, accumulate=add)
    tol = half_step(dw_dtype) * sums.abs() * (dw_dtype == BF16) + (count + 8) * U * sizes
    assert ((dW.double() - sums).abs() <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,pitch,offset", [(64, 72, 0), (64, 65, 0), (64, 80, 1), (250, 256, 2)])
def test_strided_rows(dgl, dtype, d, pitch, offset):
    """Rows apart and off their 16-byte units; nothing beside them is written."""
    T, V = 300, 120
    gen = torch.Generator(device="cuda").manual_seed(5)

    def strided(rows):
        whole = torch.full((rows * pitch + offset + 16,), 7.0, dtype=dtype, device="cuda")
        view = whole[offset:offset + rows * pitch].view(rows, pitch)[:, :d]
        view.copy_(torch.randn(rows, d, device="cuda", generator=gen))
        return whole, view

    tokens = make_tokens(T, V, "mixed")
    _, W = strided(V)
    _, dY = strided(T)
    for whole, out, call, plain in (
            (*strided(T), lambda o: dgl.embedding(tokens, W, scale=3.0, out=o),
             lambda: dgl.embedding(tokens, W.contiguous(), scale=3.0)),
            (*strided(V), lambda o: dgl.embedding_grad(tokens, dY, V, dW=o),
             lambda: dgl.embedding_grad(tokens, dY.contiguous(), V, dW=torch.empty(V, d, dtype=dtype, device="cuda")))):
        got = call(out)
        assert torch.equal(got.nan_to_num(), plain().nan_to_num())
        whole[offset:offset + len(out) * pitch].view(len(out), pitch)[:, :d] = 7.0
        assert (whole == 7.0).all()


def test_no_tokens(dgl):
    tokens = torch.empty(0, dtype=torch.int64, device="cuda")
    dY = torch.empty(0, 48, dtype=BF16, device="cuda")
    assert dgl.embedding(tokens, torch.ones(5, 48, device="cuda")).shape == (0, 48)
    assert not dgl.embedding_grad(tokens, dY, 900).any()
    dW = torch.ones(900, 48, device="cuda")
    dgl.embedding_grad(tokens, dY, 900, dW=dW, accumulate=True)
    assert (dW == 1).all()


def test_ignore_index_inside_the_vocabulary(dgl):
    """A padding token with a row of its own: zeros, and no gradient."""
    W = torch.randn(10, 32, device="cuda")
    tokens = torch.tensor([3, 0, 3, 7], device="cuda")
    Y = dgl.embedding(tokens, W, ignore_index=3)
    assert not Y[0].any() and torch.equal(Y[1], W[0])
    dW = dgl.embedding_grad(tokens, torch.ones(4, 32, device="cuda"), 10, ignore_index=3, dw_dtype=dgl.OUT_F32)
    assert not dW[3].any() and (dW[[0, 7]] == 1).all()


def test_infinities_stay_in_their_row(dgl):
    tokens = make_tokens(500, 60, "zipf")
    dY = torch.randn(500, 64, device="cuda")
    clean = dgl.embedding_grad(tokens, dY, 60, dw_dtype=dgl.OUT_F32)
    row = tokens[250].item()
    dY[250, 5] = float("inf")
    got = dgl.embedding_grad(tokens, dY, 60, dw_dtype=dgl.OUT_F32)
    assert got[row, 5] == float("inf")
    got[row, 5] = clean[row, 5]
    assert torch.equal(got, clean)


def test_streams_and_graphs(dgl):
    V, d = 5000, 256
    gen = torch.Generator(device="cuda").manual_seed(4)
    tokens = make_tokens(6000, V, "mixed")
    dY = torch.randn(6000, d, device="cuda", generator=gen).bfloat16()
    want = dgl.embedding_grad(tokens, dY, V)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [dgl.embedding_grad(tokens, dY, V, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)

    held = make_tokens(6000, V, "one")
    dW = torch.zeros(V, d, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dgl.embedding_grad(held, dY, V)
        dgl.embedding_grad(held, dY, V, dW=dW, accumulate=True)
    held.copy_(tokens)
    for k in range(1, 3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    once = dgl.embedding_grad(tokens, dY, V, dw_dtype=dgl.OUT_F32)
    assert torch.allclose(dW, 2 * once, rtol=1e-6, atol=1e-5)


def test_large_offsets(dgl):
    """Rows past 2^31 elements of W, Y and dW."""
    V, d = (1 << 31) // 4096 + 7, 4096
    W = torch.zeros(V, d, dtype=BF16, device="cuda")
    W[-3:] = 1.5
    tokens = torch.tensor([V - 1, 0, V - 2, V - 1], device="cuda")
    Y = dgl.embedding(tokens, W)
    assert (Y[[0, 2, 3]] == 1.5).all() and not Y[1].any()
    dW = dgl.embedding_grad(tokens, Y, V, dW=W)
    assert dW is W and (dW[-1] == 3.0).all() and (dW[-2] == 1.5).all() and not dW[-3].any() and not dW[:4].any()
