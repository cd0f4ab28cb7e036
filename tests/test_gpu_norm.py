"""Layer norm and its gradient against their definitions in fp64.

u is fp32's unit roundoff.  A row's sums take at most 16 additions in a thread
and 10 across threads (or d / 512 and 26 past 16384), so a statistic is off by less than 64 u
of the sum of magnitudes (128 u past 16384); rounding to the output's type adds half a step.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0**-24
EPS = 1e-5


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


def half_step(t):
    return torch.finfo(t).eps / 2


def make(rows, d, dtype, w_dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    x = (normal(rows, d) * torch.exp(0.5 * normal(rows, 1)) + normal(rows, 1)).to(dtype)
    dy = normal(rows, d).to(dtype)
    if w_dtype is None:
        return x, dy, None, None
    return x, dy, (1 + 0.2 * normal(d)).to(w_dtype), normal(d).to(w_dtype)


def forward64(x, w, b):
    x = x.double()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = (c.square().mean(1) + EPS).rsqrt()
    h = c * rstd[:, None]
    wd = 1.0 if w is None else w.double()
    bd = 0.0 if b is None else b.double()
    return h * wd + bd, mean, rstd, h


def check(name, got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    if bad.any():
        at = bad.nonzero()[0].tolist()
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {at}: "
                             f"{got[tuple(at)].item()} for {want[tuple(at)].item()}")


SHAPES = [(1, 1), (1, 8), (3, 7), (5, 16), (130, 17), (257, 24), (64, 100), (33, 129), (300, 512), (77, 513),
          (40, 1023), (9, 1024), (700, 1025), (6, 2048), (2100, 768), (19, 4096), (3, 4100), (11, 8191), (5, 8192),
          (4, 8194), (7, 12288), (3, 16383), (2, 16384), (3, 16392), (2, 20001), (1300, 4096), (400, 8200),
          (333, 12288), (700, 16400), (5000, 40), (90000, 8)]
TYPES = [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16), (BF16, None)]


@pytest.mark.parametrize("dtype,w_dtype", TYPES)
@pytest.mark.parametrize("rows,d", SHAPES)
def test_forward_and_gradient(dgl, rows, d, dtype, w_dtype):
    x, dy, w, b = make(rows, d, dtype, w_dtype)
    k = 128 if d > 16384 else 64
    y, mean, rstd = dgl.layer_norm(x, w, b, eps=EPS)
    want, mean64, rstd64, h = forward64(x, w, b)
    size = x.double().abs()
    average = size.mean(1)
    check("mean", mean, mean64, k * U * average)
    # the mean's error enters the variance squared
    check("rstd", rstd, rstd64, rstd64 * (k * U + (k * U * average * rstd64).square()))
    wd = torch.ones(d, dtype=torch.float64, device="cuda") if w is None else w.double()
    bd = torch.zeros_like(wd) if b is None else b.double()
    reach = (size + average[:, None]) * rstd64[:, None]
    check("y", y, want, half_step(dtype) * want.abs() + k * U * (reach * wd.abs() + bd.abs()) + 1e-30)

    dx, dw, db = dgl.layer_norm_grad(dy, x, mean, rstd, w)
    # the gradient is the formula's at the statistics given
    mean64, rstd64 = mean.double()[:, None], rstd.double()[:, None]
    g = dy.double()
    h = (x.double() - mean64) * rstd64
    eh = 4 * U * (size + mean64.abs()) * rstd64
    u = g * wd
    s, q = u.mean(1, keepdim=True), (u * h).mean(1, keepdim=True)
    want = rstd64 * (u - s - h * q)
    tol = half_step(dtype) * want.abs() + k * U * rstd64 * (u.abs() + u.abs().mean(1, keepdim=True)
                                                            + h.abs() * (u * h).abs().mean(1, keepdim=True))
    tol += 2 * rstd64 * (eh * q.abs() + h.abs() * (u.abs() * eh).mean(1, keepdim=True))
    check("dx", dx, want, tol + 1e-30)
    check("dw", dw, (g * h).sum(0), (rows + 64) * U * (g * h).abs().sum(0) + (g.abs() * eh).sum(0) + 1e-30)
    check("db", db, g.sum(0), (rows + 64) * U * g.abs().sum(0) + 1e-30)
    # equal calls give equal bits
    again = dgl.layer_norm_grad(dy, x, mean, rstd, w)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))
    assert dgl.device_status() == dgl.DGL_OK


def test_gradient_against_differences(dgl):
    """In fp32 on a small row, against central differences of the fp64 formula."""
    x, dy, w, b = make(3, 40, F32, F32)
    y, mean, rstd = dgl.layer_norm(x, w, b, eps=EPS)
    dx, dw, db = dgl.layer_norm_grad(dy, x, mean, rstd, w)

    def loss(x, w, b):
        c = x - x.mean(1, keepdim=True)
        return ((c * (c.square().mean(1, keepdim=True) + EPS).rsqrt() * w + b) * dy.double()).sum()

    leaves = [t.double() for t in (x, w, b)]
    step = 1e-5
    for i, got in enumerate((dx, dw, db)):
        for at in range(0, leaves[i].numel(), 7):
            moved = [t.clone() for t in leaves]
            moved[i].view(-1)[at] += step
            up = loss(*moved)
            moved[i].view(-1)[at] -= 2 * step
            slope = (up - loss(*moved)) / (2 * step)
            # differences: step^2 of the third derivative; fp32: as above
            assert abs(got.view(-1)[at].item() - slope.item()) < 1e-4 * (1 + abs(slope.item()))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d,pitch,offset", [(64, 72, 0), (64, 65, 0), (64, 80, 1), (1000, 1001, 3), (2048, 2056, 8)])
def test_strided_rows(dgl, dtype, d, pitch, offset):
    """Rows apart and off their 16-byte units; nothing beside them is written."""
    rows = 37
    x0, dy0, w, b = make(rows, d, dtype, F32)

    def strided(t):
        whole = torch.full((rows * pitch + offset + 16,), 7.0, dtype=dtype, device="cuda")
        view = whole[offset:offset + rows * pitch].view(rows, pitch)[:, :d]
        view.copy_(t)
        return whole, view

    _, x = strided(x0)
    _, dy = strided(dy0)
    whole, out = strided(x0)
    y, mean, rstd = dgl.layer_norm(x, w, b, out=out)
    want, mean1, rstd1 = dgl.layer_norm(x0, w, b)
    assert y is out
    tol = half_step(dtype) * 2 + 64 * U
    assert torch.allclose(y.double(), want.double(), rtol=tol, atol=1e-5)
    guard = whole.clone()
    guard[offset:offset + rows * pitch].view(rows, pitch)[:, :d] = 7.0
    assert (guard == 7.0).all()
    got = dgl.layer_norm_grad(dy, x, mean, rstd, w)
    want = dgl.layer_norm_grad(dy0, x0, mean1, rstd1, w)
    for p, q in zip(got, want):
        assert torch.allclose(p.double(), q.double(), rtol=2 * half_step(p.dtype) + 1e-5, atol=1e-4)


@pytest.mark.parametrize("d", [64, 1024, 8192, 12288])
@pytest.mark.parametrize("w_dtype", [BF16, F32])
def test_weights_off_their_units(dgl, d, w_dtype):
    """Weights and biases that begin anywhere, beside rows that are whole units; a norm without one of them."""
    x, dy, w, b = make(200, d, BF16, w_dtype)
    w1, b1 = torch.cat([w[:1], w])[1:], torch.cat([b[:3], b])[3:]
    assert w1.data_ptr() % 16 and torch.equal(w1, w)
    want, got = dgl.layer_norm(x, w, b), dgl.layer_norm(x, w1, b1)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    want = dgl.layer_norm_grad(dy, x, want[1], want[2], w)
    got = dgl.layer_norm_grad(dy, x, got[1], got[2], w1)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    ones, zeros = torch.ones_like(w), torch.zeros_like(b)
    assert torch.equal(dgl.layer_norm(x, None, b)[0], dgl.layer_norm(x, ones, b)[0])
    assert torch.equal(dgl.layer_norm(x, w)[0], dgl.layer_norm(x, w, zeros)[0])


@pytest.mark.parametrize("d", [96, 1000, 9000])
def test_in_place(dgl, d):
    x, _, w, b = make(50, d, BF16, F32)
    want = dgl.layer_norm(x, w, b)
    got = dgl.layer_norm(x, w, b, out=x)
    assert got[0] is x and all(torch.equal(p, q) for p, q in zip(got, want))


def test_constant_rows_and_bad_rows(dgl):
    """A constant row is its bias; NaN and infinities stay in their own row."""
    x, dy, w, b = make(9, 520, F32, F32)
    x[2] = 3.0
    x[4, 7], x[6, 3] = float("nan"), float("inf")
    y, mean, rstd = dgl.layer_norm(x, w, b, eps=EPS)
    assert torch.equal(y[2], b) and mean[2] == 3.0
    assert abs(rstd[2].item() - EPS**-0.5) < 1e-4 * EPS**-0.5
    assert y[4].isnan().all() and y[6].isnan().all()
    keep = [0, 1, 2, 3, 5, 7, 8]
    clean = dgl.layer_norm(x[keep], w, b, eps=EPS)
    assert torch.equal(y[keep], clean[0])
    dx, _, _ = dgl.layer_norm_grad(dy, x, mean, rstd, w)
    assert dx[4].isnan().all() and dx[keep].isfinite().all()


@pytest.mark.parametrize("d", [48, 1500, 10000])
def test_large_offset(dgl, d):
    """A mean a thousand times the spread: the variance is no difference of large sums."""
    x = 1000.0 + torch.randn(20, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    _, mean, rstd = dgl.layer_norm(x, eps=0.0)
    _, mean64, _, _ = forward64(x, None, None)
    true = 1.0 / (x.double() - mean64[:, None]).square().mean(1).sqrt()
    # a mean off by 64 u x 1000 moves the variance by its square, 1.5e-5 at most
    assert ((rstd.double() - true).abs() <= 3e-5 * true).all()


@pytest.mark.parametrize("rows,d", [(0, 64), (1, 64), (333, 1023), (4, 9000), (3, 17000)])
@pytest.mark.parametrize("dw_dtype", ["bf16", "fp32"])
def test_gradient_parts(dgl, rows, d, dw_dtype):
    """Each gradient alone, of either type, added or not; no rows."""
    x, dy, w, b = make(rows, d, BF16, F32)
    code = dgl.OUT_BF16 if dw_dtype == "bf16" else dgl.OUT_F32
    _, mean, rstd = dgl.layer_norm(x, w, b)
    dx, dw, db = dgl.layer_norm_grad(dy, x, mean, rstd, w, dw_dtype=code)
    assert dw.dtype == db.dtype == (BF16 if dw_dtype == "bf16" else F32)
    if rows == 0:
        assert not dw.any() and not db.any()
    alone = dgl.layer_norm_grad(dy, x, mean, rstd, w, need_dw=False, need_db=False)
    assert torch.equal(alone[0], dx) and alone[1] is None and alone[2] is None
    alone = dgl.layer_norm_grad(dy, x, mean, rstd, w, need_dx=False, need_db=False, dw_dtype=code)
    assert alone[0] is None and torch.equal(alone[1], dw) and alone[2] is None
    alone = dgl.layer_norm_grad(dy, x, mean, rstd, w, need_dx=False, need_dw=False, dw_dtype=code)
    assert torch.equal(alone[2], db)
    if dw_dtype == "fp32":
        a, c = torch.full_like(dw, 2.0), torch.full_like(db, -3.0)
        dgl.layer_norm_grad(dy, x, mean, rstd, w, dweight=a, dbias=c, accumulate=True)
        assert torch.equal(a, dw + 2.0) and torch.equal(c, db - 3.0)


def test_streams_and_graphs(dgl):
    """Two streams at once with workspaces of their own; a captured pass replayed on new inputs."""
    x, dy, w, b = make(600, 2048, BF16, F32)
    y, mean, rstd = dgl.layer_norm(x, w, b)
    want = (y, *dgl.layer_norm_grad(dy, x, mean, rstd, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in streams:
            out = dgl.layer_norm(x, w, b, stream=s)
            got.append((out[0], *dgl.layer_norm_grad(dy, x, out[1], out[2], w, stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for g in got for p, q in zip(g, want))

    held = [torch.zeros_like(x), torch.zeros_like(dy)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dgl.layer_norm(held[0], w, b)
        out = (out[0], *dgl.layer_norm_grad(held[1], held[0], out[1], out[2], w))
    for _ in range(2):
        held[0].copy_(x)
        held[1].copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, want))
        held[0].zero_()
        graph.replay()


def test_many_rows(dgl):
    """Offsets past 2^31 elements."""
    rows, d = (1 << 31) // 4096 + 5, 4096
    x = torch.zeros(rows, d, dtype=BF16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x[-4:] = torch.randn(4, d, device="cuda", generator=gen).bfloat16()
    y, mean, rstd = dgl.layer_norm(x, out=x.clone())
    last = dgl.layer_norm(x[-4:].clone())
    assert torch.equal(y[-4:], last[0]) and not y[:64].any()
    dx, dw, _ = dgl.layer_norm_grad(x, x, mean, rstd)
    want = dgl.layer_norm_grad(x[-4:].clone(), x[-4:].clone(), mean[-4:].clone(), rstd[-4:].clone())
    assert torch.equal(dx[-4:], want[0])
    assert torch.allclose(dw, want[1], rtol=1e-5, atol=1e-5)
