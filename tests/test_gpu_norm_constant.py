"""Layer norm of rows whose elements are equal, or nearly so beside their size: h is zero there, or as exact as the
fp32 mean allows."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0**-24
EPS = 1e-5
# a part of a warp, a warp, several, a ragged number; past 8192; past 16384; rows off their units
WIDTHS = [1, 8, 48, 333, 512, 1000, 1023, 1024, 4100, 8191, 12288, 12287, 16400]
VALUES = [3.0, -100.5, 1000.0, 2992.0, 30000.0, -1e30, 1e-30, 0.0]


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


def half_step(t):
    return torch.finfo(t).eps / 2


def rows_of(values, d, dtype):
    return torch.tensor(values, device="cuda").to(dtype)[:, None].repeat(1, d)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", WIDTHS)
def test_equal_elements(dgl, dtype, d):
    """The mean is the element, y is the bias, and the row adds nothing to dweight; dx is that of h = 0."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    values = VALUES + ([1000.1, 0.3, 2.9999998] if dtype == F32 else [])
    x = rows_of(values, d, dtype)
    w, b = torch.randn(d, device="cuda", generator=gen), torch.randn(d, device="cuda", generator=gen)
    dy = torch.randn(len(values), d, device="cuda", generator=gen).to(dtype)
    y, mean, rstd = dgl.layer_norm(x, w, b, eps=EPS)
    assert torch.equal(mean, x[:, 0].float())
    assert ((rstd.double() - EPS**-0.5).abs() <= 4 * U * EPS**-0.5).all()
    # what the first mean is off by, 64 u of the element at most, is taken away to within 4 u of itself
    off = 256 * U * U * x.double().abs() * rstd.double()[:, None] * w.double().abs()
    assert ((y.double() - b.double()).abs() <= (half_step(dtype) + U) * (b.double().abs() + off) + off).all()
    dx, dw, db = dgl.layer_norm_grad(dy, x, mean, rstd, w)
    assert not dw.any()
    u = dy.double() * w.double()
    want = rstd.double()[:, None] * (u - u.mean(1, keepdim=True))
    tol = half_step(dtype) * want.abs() + 128 * U * rstd.double()[:, None] * (u.abs() + u.abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype,size,spread", [(BF16, 1000.0, 4.0), (BF16, 30000.0, 128.0), (F32, 1000.0, 0.01),
                                               (F32, 30000.0, 1.0)])
@pytest.mark.parametrize("d", [48, 333, 1000, 1024, 4100, 12288, 12287, 16400])
def test_little_spread(dgl, dtype, size, spread, d):
    """Rows of two neighbouring values at a large size: y, and dweight from the statistics kept."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = (size + spread * torch.randint(0, 2, (40, d), device="cuda", generator=gen)).to(dtype)
    dy = torch.randn(40, d, device="cuda", generator=gen).to(dtype)
    y, mean, rstd = dgl.layer_norm(x, eps=EPS)
    x64 = x.double()
    mean64 = x64.mean(1, keepdim=True)
    c = x64 - mean64
    rstd64 = (c.square().mean(1, keepdim=True) + EPS).rsqrt()
    # the mean is rounded once, beside 64 u (past 16384 128 u) of what the elements are away from it
    k = 128 if d > 16384 else 64
    away = c.abs().mean(1)
    off = U * mean64[:, 0].abs() + k * U * away
    assert ((mean.double() - mean64[:, 0]).abs() <= off).all()
    assert ((rstd.double() - rstd64[:, 0]).abs() <= rstd64[:, 0] * (k * U + (off * rstd64[:, 0]).square())).all()
    # y is taken from the mean before it is rounded
    h = c * rstd64
    reach = (c.abs() + away[:, None]) * rstd64
    assert ((y.double() - h).abs() <= half_step(dtype) * h.abs() + 2 * k * U * reach + k * U * U * size * rstd64).all()
    dw = dgl.layer_norm_grad(dy, x, mean, rstd, need_dx=False, need_db=False)[1]
    g = dy.double()
    kept = (x64 - mean.double()[:, None]) * rstd.double()[:, None]
    assert ((dw.double() - (g * kept).sum(0)).abs() <= (40 + 64) * U * (g * kept).abs().sum(0) + 1e-30).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [48, 1000, 4100, 12288, 16400])
def test_rows_that_are_not_finite(dgl, dtype, d):
    """An infinite element makes its row's mean infinite and its y NaN, wherever it stands."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(6, d, device="cuda", generator=gen).to(dtype)
    clean = dgl.layer_norm(x)
    inf = float("inf")
    x[0, 0], x[1, d - 1], x[2, d // 2], x[3, 0], x[3, d - 1] = inf, -inf, float("nan"), inf, -inf
    y, mean, _ = dgl.layer_norm(x)
    assert mean[0] == inf and mean[1] == -inf and mean[2:4].isnan().all()
    assert y[:4].isnan().all()
    assert all(torch.equal(p[4:], q[4:]) for p, q in zip((y, mean), clean))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("d", [1, 48, 333, 1000, 1024, 4100, 12288, 12287, 16400])
@pytest.mark.parametrize("size", [1e20, 1e25, 1e28, 1e33])
def test_squares_past_fp32(dgl, dtype, d, size):
    """Where the squares overflow, the variance is infinite: rstd is zero and y the bias."""
    gen = torch.Generator(device="cuda").manual_seed(d)
    b = torch.randn(d, device="cuda", generator=gen)
    spread = (size * torch.randn(5, d, device="cuda", generator=gen)).to(dtype)
    if d == 1:  # a row of one element has none
        y, _, rstd = dgl.layer_norm(spread, None, b, eps=EPS)
        assert torch.equal(y, b.to(dtype).expand(5, 1)) and ((rstd - EPS**-0.5).abs() <= 4 * U * EPS**-0.5).all()
        return
    for x in (spread, (size * (1 + torch.randint(0, 2, (5, d), device="cuda", generator=gen) / 8)).to(dtype)):
        y, mean, rstd = dgl.layer_norm(x, None, b, eps=EPS)
        assert not rstd.any() and torch.equal(y, b.to(dtype).expand(5, d))
        mean64 = x.double().mean(1)
        assert ((mean.double() - mean64).abs() <= 128 * U * x.double().abs().mean(1)).all()
