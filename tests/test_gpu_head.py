"""The losses of a linear head (linear_cross_entropy, linear_distill) against
their definitions in 64 bits.

Tolerances.  With u = 2^-24 and a product of d terms accumulated by the tensor
core in steps of 16, each step losing at most 4 u of the running magnitude, a
logit is off by at most
    ez = (d / 16 + 4) 4 u |s| max_v sum_k |x_k w_vk|
and the normaliser by ez plus 2^-20 (1 + |lse|) for the exponentials, sums
and the logarithm; a loss by 2 ez + 2^-20 (1 + |lse| + max_k |z_k| + max |log q|).
A gradient entry dz = g (Q p - q) is rounded to bf16 at most twice, its factor
of the row once more (3 x 2^-9 relative), and p carries the logits' error:
    |d dz| <= |dz| (3 x 2^-9 + 2^-13) + |g| Q p (2 ez + 2^-17) + |g| q 2^-20
so dX is off by s |d dz| |W| plus 2^-8 of itself (its own rounding, and the
fp32 sums of the product), dW by s |d dz|^T |X| plus the same.
"""
import math

import pytest
import torch

import dense_gemm_linear_gb300 as dgl

pytestmark = pytest.mark.gpu
DEV = "cuda"
IGNORE = -100


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _inputs(T, V, d, seed=0, w_std=0.05):
    g = _gen(seed)
    X = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    W = (w_std * torch.randn(V, d, device=DEV, generator=g)).bfloat16()
    target = torch.randint(0, V, (T,), device=DEV, generator=g)
    if T:
        X = (X.float() + 6.0 * torch.rand(T, 1, device=DEV, generator=g) * W[target].float()
             / (W[target].float().norm(dim=1, keepdim=True).square() + 1e-3)).bfloat16()
    grad = (torch.rand(T, device=DEV, generator=g) - 0.2).float()
    return X, W, target, grad


def _wanted_xent(T, V, target, ignore=IGNORE):
    """The asked-for distribution [T, V], sum q log q, and which rows have one."""
    q = torch.zeros(T, V, dtype=torch.float64, device=DEV)
    live = target != ignore
    r = torch.nonzero(live)[:, 0]
    q[r, target[r]] = 1.0
    return q, torch.zeros(T, dtype=torch.float64, device=DEV), live, 0.0


def _wanted_distill(T, V, indices, logits, temp, teacher_lse=None):
    q = torch.zeros(T, V, dtype=torch.float64, device=DEV)
    qlogq = torch.zeros(T, dtype=torch.float64, device=DEV)
    live = torch.zeros(T, dtype=torch.bool, device=DEV)
    big = 0.0
    for t in range(T):
        keep = [j for j in range(indices.shape[1])
                if indices[t, j].item() >= 0 and logits[t, j].item() != -math.inf]
        if not keep:
            continue
        live[t] = True
        l = logits[t, keep].double() / temp
        lq = l - (torch.logsumexp(l, 0) if teacher_lse is None else teacher_lse[t].double())
        q[t].index_add_(0, indices[t, keep], lq.exp())
        qlogq[t] = torch.special.xlogy(lq.exp(), lq.exp()).sum()
        big = max(big, lq.abs().max().item())
    return q, qlogq, live, big


def _check(X, W, scale, wanted, grad, got, dw_before=None, ignored_rows=None):
    """Compares (loss, lse[, dX, dW]) with the definitions."""
    T, d = X.shape
    q, qlogq, live, big = wanted
    x, w = X.double(), W.double()
    if ignored_rows is not None:
        x = torch.where(ignored_rows[:, None], 0.0, x)
    z = scale * (x @ w.T)
    ez = ((d / 16 + 4) * 4 * 2.0**-24) * abs(scale) * (x.abs() @ w.abs().T).amax(1)
    lse = torch.logsumexp(z, 1)
    Q = q.sum(1)
    loss = torch.where(live, qlogq - (q * z).sum(1) + Q * lse, 0.0)
    at = torch.where(q > 0, z.abs(), 0.0).amax(1)
    ok_rows = torch.ones(T, dtype=torch.bool, device=DEV) if ignored_rows is None else ~ignored_rows
    e_lse = ez + 2.0**-20 * (1 + lse.abs())
    assert (((got[1].double() - lse).abs() <= e_lse) | ~ok_rows).all(), \
        f"lse off by {(got[1].double() - lse).abs().max().item():.3g}"
    e_loss = (1 + Q) * (2 * ez + 2.0**-20 * (1 + lse.abs() + at + big))
    bad = ~((got[0].double() - loss).abs() <= torch.where(live, e_loss, torch.zeros_like(e_loss)))
    assert not bad.any(), f"loss of rows {torch.nonzero(bad)[:5, 0].tolist()}: {got[0][bad][:5]} for {loss[bad][:5]}"
    if grad is None:
        assert len(got) == 2
        return
    p = torch.exp(z - lse[:, None])
    g = torch.where(live, grad.double(), 0.0)[:, None]
    dz = g * (Q[:, None] * p - q)
    e_dz = dz.abs() * (3 * 2.0**-9 + 2.0**-13) + g.abs() * Q[:, None] * p * (2 * ez[:, None] + 2.0**-17) \
        + g.abs() * q * 2.0**-20
    for name, have, ref, err in (("dX", got[2], scale * (dz @ w), abs(scale) * (e_dz @ w.abs())),
                                 ("dW", got[3], scale * (dz.T @ x), abs(scale) * (e_dz.T @ x.abs()))):
        if have is None:
            continue
        if name == "dW" and dw_before is not None:
            ref = ref + dw_before.double()
        tol = err + 2.0**-8 * ref.abs() + 1e-30
        off = (have.double() - ref).abs()
        bad = ~(off <= tol)
        assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {off[bad].max().item():.3g} where "
                               f"{tol[bad].max().item():.3g} is allowed, first at {torch.nonzero(bad)[0].tolist()}")


def _status():
    st = dgl.device_status()
    assert st == dgl.DGL_OK, dgl.status_string(st)


SIZES = [(1, 1, 8), (1, 7, 8), (1, 257, 64), (2, 1000, 72), (5, 31, 2048), (16, 11007, 128), (127, 129, 136),
         (128, 256, 64), (129, 513, 264), (257, 1000, 512), (300, 50257, 64), (33, 4095, 512), (640, 3001, 320),
         (1100, 2048, 128)]


@pytest.mark.parametrize("T,V,d", SIZES)
@pytest.mark.parametrize("with_grad", [False, True])
def test_xent_sizes(T, V, d, with_grad):
    X, W, target, grad = _inputs(T, V, d)
    target[::7] = IGNORE
    if T == 1:
        target[0] = V - 1
    g = grad if with_grad else None
    got = dgl.linear_cross_entropy(X, W, target, g)
    _status()
    _check(X, W, 1.0, _wanted_xent(T, V, target), g, got)


@pytest.mark.parametrize("seed", range(6))
def test_xent_drawn_sizes(seed):
    import random
    r = random.Random(seed)
    T, V, d = r.randint(1, 900), r.randint(1, 6000), 8 * r.randint(1, 60)
    X, W, target, grad = _inputs(T, V, d, seed)
    scale = r.choice([1.0, 0.5, -1.5])
    got = dgl.linear_cross_entropy(X, W, target, grad, logit_scale=scale)
    _status()
    _check(X, W, scale, _wanted_xent(T, V, target), grad, got)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_xent_all_rows_ignored(T):
    X, W, target, grad = _inputs(T, 515, 64)
    target.fill_(7)
    got = dgl.linear_cross_entropy(X, W, target, grad, ignore_index=7)
    _status()
    assert (got[0] == 0).all() and (got[2] == 0).all() and (got[3] == 0).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_xent_ignored_rows_do_not_leak(value):
    T, V, d = 200, 777, 72
    X, W, target, grad = _inputs(T, V, d)
    ignored = torch.zeros(T, dtype=torch.bool, device=DEV)
    ignored[[0, 31, 130, 199]] = True
    target[ignored] = IGNORE
    X[ignored] = value
    got = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    assert (got[2][ignored] == 0).all()
    _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got, ignored_rows=ignored)


@pytest.mark.parametrize("wrong", [-1, 777, 2**31, 2**40, -2**33])
def test_xent_target_out_of_range(wrong):
    T, V, d = 150, 777, 64
    X, W, target, grad = _inputs(T, V, d)
    target[5] = wrong
    got = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    assert got[0][5].isnan() and (got[2][5] == 0).all()
    # for the rest it is a row without a target
    clean = target.clone()
    clean[5] = IGNORE
    loss = got[0].clone()
    loss[5] = 0
    _check(X, W, 1.0, _wanted_xent(T, V, clean), grad, (loss,) + got[1:])


def test_xent_nan_stays_in_its_row():
    T, V, d = 140, 600, 64
    X, W, target, grad = _inputs(T, V, d)
    X[9, 3] = float("nan")
    loss, lse, dX, _ = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    others = torch.arange(T, device=DEV) != 9
    assert loss[9].isnan() and lse[9].isnan()
    assert not loss[others].isnan().any() and not dX[others].isnan().any()


@pytest.mark.parametrize("offset", [-300.0, -60.0, 60.0, 300.0])
def test_xent_common_offset(offset):
    """All logits of a row moved by the same large amount: the softmax does not change."""
    T, V, d = 90, 700, 64
    X, W, target, grad = _inputs(T, V, d)
    W[:, 0] = 8.0
    X[:, 0] = offset / 8.0
    got = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)


@pytest.mark.parametrize("spread", [10.0, 60.0, 400.0])
@pytest.mark.parametrize("V", [130, 700, 5000])
def test_xent_wide_logits(spread, V):
    """Logits spread far beyond what one exponential can hold, with the target
    among the lowest, the highest, or alone: some rows' maxima lie in a
    later or earlier part of the vocabulary than their targets."""
    T, d = 160, 64
    X, W, target, grad = _inputs(T, V, d, w_std=0.01)
    W[:, 1] = torch.linspace(-1, 1, V, device=DEV).bfloat16()
    X[:, 1] = spread * torch.linspace(-1, 1, T, device=DEV).bfloat16()
    target[:] = torch.randint(0, V, (T,), device=DEV, generator=_gen(3))
    target[:20] = 0
    target[-20:] = 0
    target[20:40] = V - 1
    target[-40:-20] = V - 1
    got = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)


@pytest.mark.parametrize("T,V", [(90, 700), (300, 2500)])
@pytest.mark.parametrize("size", [2.0**10, 2.0**17, 2.0**24, 2.0**30])
def test_xent_huge_logits(size, T, V):
    """Logits so large that their own last bit is worth more than a factor of
    two: each is one exact product, and what is next to the largest is either
    equal to it or at least 2^-9 of it lower, so the answer is still sharp."""
    d = 64
    _, W, target, grad = _inputs(T, V, d)
    W = torch.where(W == 0, 0.25, W.float().sign() * (0.25 + W.float().abs())).bfloat16()
    rows = torch.arange(T, device=DEV)
    X = torch.zeros(T, d, device=DEV)
    X[rows, rows % d] = torch.where(rows % 3 == 0, -size, size)
    X = X.bfloat16()
    x, w = X.double(), W.double()
    z = x @ w.T
    high = z.amax(1, keepdim=True)
    target = torch.where(rows % 2 == 0, z.argmax(1), target)
    loss, lse, dX, dW = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    p = torch.softmax(z, 1)
    rest = torch.where(z < high, p, 0.0)
    q = torch.zeros_like(p).scatter_(1, target[:, None], 1.0)
    # y = z log2(e) is rounded once, the difference of two of them carries both
    ez = 2.0**-23 * z.abs().amax(1, keepdim=True)
    want = torch.logsumexp(z, 1)
    assert ((lse.double() - want).abs() <= 2.0**-20 * (1 + want.abs())).all()
    at = z.gather(1, target[:, None])
    short = (high - at + (p.sum(1, keepdim=True) / p.amax(1, keepdim=True)).log())[:, 0]
    e_loss = 2.0**-20 * (1 + short) + torch.where(at < high, 2 * ez, 0.0)[:, 0] + (2 * ez * rest.sum(1, keepdim=True))[:, 0]
    assert ((loss.double() - short).abs() <= e_loss).all()
    g = grad.double()[:, None]
    dz = g * (p - q)
    e_dz = dz.abs() * (3 * 2.0**-9 + 2.0**-13) + g.abs() * (p * 2.0**-17 + q * 2.0**-20 + 2.0**-40) \
        + g.abs() * 2 * ez * (rest + p * rest.sum(1, keepdim=True))
    for have, ref, err in ((dX, dz @ w, e_dz @ w.abs()), (dW, dz.T @ x, e_dz.T @ x.abs())):
        assert ((have.double() - ref).abs() <= err + 2.0**-8 * ref.abs() + 1e-30).all()


def test_xent_sure_rows():
    """Targets with probability close to one: the gradient is the small rest."""
    T, V, d = 64, 400, 128
    X, W, target, grad = _inputs(T, V, d)
    w = W[target].float()
    X = (w * torch.linspace(4, 40, T, device=DEV)[:, None] / w.square().sum(1, keepdim=True)).bfloat16()
    got = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)


@pytest.mark.parametrize("T,V,d", [(2, 46, 128), (1, 1306, 440), (94, 3000, 1000), (207, 2600, 376)])
def test_xent_probabilities_down_to_nothing(T, V, d):
    """Logits spread over hundreds: an entry below 2^-40 of the largest of its 128
    columns may count as zero, so dz is also off by up to 2^-40 |g| an entry."""
    X, W, target, grad = _inputs(T, V, d, w_std=0.5)
    loss, lse, dX, dW = dgl.linear_cross_entropy(X, W, target, grad, logit_scale=3.0)
    _status()
    _check(X, W, 3.0, _wanted_xent(T, V, target), None, (loss, lse))
    x, w = X.double(), W.double()
    z = 3.0 * (x @ w.T)
    ez = ((d / 16 + 4) * 4 * 2.0**-24) * 3.0 * (x.abs() @ w.abs().T).amax(1)
    p = torch.softmax(z, 1)
    g = grad.double()[:, None]
    dz = g * (p - torch.zeros_like(p).scatter_(1, target[:, None], 1.0))
    e_dz = dz.abs() * (3 * 2.0**-9 + 2.0**-13) + g.abs() * p * (2 * ez[:, None] + 2.0**-17) + g.abs() * 2.0**-40
    # (the target's entry carries the rounding of its own sum of the others)
    e_dz.scatter_add_(1, target[:, None], g.abs() * 2.0**-20)
    for have, ref, err in ((dX, dz @ w, e_dz @ w.abs()), (dW, dz.T @ x, e_dz.T @ x.abs())):
        assert ((have.double() - 3.0 * ref).abs() <= 3.0 * err + 2.0**-8 * (3.0 * ref).abs() + 1e-30).all()


def test_strides_and_untouched_padding():
    T, V, d = 150, 999, 72
    X, W, target, grad = _inputs(T, V, d)
    Xp = torch.full((T, d + 24), float("nan"), device=DEV, dtype=torch.bfloat16)
    Wp = torch.full((V, d + 8), float("nan"), device=DEV, dtype=torch.bfloat16)
    Xp[:, :d], Wp[:, :d] = X, W
    for dt in (torch.bfloat16, torch.float32):
        dWp = torch.full((V + 2, d + 16), 7.0, device=DEV, dtype=dt)
        got = dgl.linear_cross_entropy(Xp[:, :d], Wp[:, :d], target, grad, dW=dWp[:V, :d])
        _status()
        _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)
        assert (dWp[V:] == 7.0).all() and (dWp[:V, d:] == 7.0).all()
    # every other row of X
    Xs = torch.zeros(2 * T, d, device=DEV, dtype=torch.bfloat16)
    Xs[::2] = X
    got = dgl.linear_cross_entropy(Xs[::2], W, target, grad)
    _status()
    _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)


@pytest.mark.parametrize("need", [(True, False), (False, True)])
def test_one_of_the_gradients(need):
    T, V, d = 140, 1000, 64
    X, W, target, grad = _inputs(T, V, d)
    got = dgl.linear_cross_entropy(X, W, target, grad, need_dx=need[0], need_dw=need[1])
    _status()
    assert (got[2] is not None) == need[0] and (got[3] is not None) == need[1]
    if need[0]:
        got = got[:3] + (None,)
        _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)
    else:
        full = dgl.linear_cross_entropy(X, W, target, grad)
        assert torch.equal(full[3], got[3])


def _workspace(T, V, d, k, dw_dtype):
    h = dgl.HeadDesc()
    h.T, h.V, h.d, h.grad, h.dX, h.dW, h.dw_dtype = T, V, d, 1, 1, 1, dw_dtype
    return dgl.dgl_head_workspace(h, k)


@pytest.mark.parametrize("dw_dtype", [dgl.OUT_BF16, dgl.OUT_F32])
@pytest.mark.parametrize("T", [128, 129, 400, 700])
def test_small_workspace_takes_chunks(T, dw_dtype):
    V, d = 1111, 96
    X, W, target, grad = _inputs(T, V, d)
    low, best = _workspace(T, V, d, 0, dw_dtype)
    assert low <= best or T <= 128
    for size in (low, (low + best) // 2, best, best + 4096):
        if size < low:
            continue
        buf = torch.full((size + 256,), 255, dtype=torch.uint8, device=DEV)  # NaN whatever type is read
        got = dgl.linear_cross_entropy(X, W, target, grad, dw_dtype=dw_dtype, workspace=buf[:size])
        _status()
        assert (buf[size:] == 255).all(), "wrote past the workspace"
        _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)


@pytest.mark.parametrize("T", [90, 300])
def test_accumulate(T):
    V, d = 650, 80
    X, W, target, grad = _inputs(T, V, d)
    before = torch.randn(V, d, device=DEV, generator=_gen(9)) * 0.05
    low, _ = _workspace(T, V, d, 0, dgl.OUT_F32)
    for ws in (None, torch.empty(low, dtype=torch.uint8, device=DEV)):
        dW = before.clone()
        got = dgl.linear_cross_entropy(X, W, target, grad, dW=dW, accumulate=True, workspace=ws)
        _status()
        assert got[3] is dW
        _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got, dw_before=before)


def test_no_tokens():
    X, W, target, grad = _inputs(0, 300, 64)
    loss, lse = dgl.linear_cross_entropy(X, W, target)
    assert loss.numel() == 0 and lse.numel() == 0
    dW = torch.full((300, 64), 3.0, device=DEV)
    dgl.linear_cross_entropy(X, W, target, grad, dW=dW, accumulate=True)
    assert (dW == 3.0).all()
    _, _, dX, dW = dgl.linear_cross_entropy(X, W, target, grad, dW=dW)
    assert dX.shape == (0, 64) and (dW == 0).all()


def test_same_inputs_give_the_same_bits():
    T, V, d = 700, 5003, 256
    X, W, target, grad = _inputs(T, V, d)
    a = dgl.linear_cross_entropy(X, W, target, grad)
    for _ in range(3):
        b = dgl.linear_cross_entropy(X, W, target, grad)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_other_stream_and_graph():
    T, V, d = 260, 2049, 128
    X, W, target, grad = _inputs(T, V, d)
    ref = dgl.linear_cross_entropy(X, W, target, grad)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = dgl.linear_cross_entropy(X, W, target, grad, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = dgl.linear_cross_entropy(X, W, target, grad)
    X2, _, target2, _ = _inputs(T, V, d, 5)
    X.copy_(X2)
    target.copy_(target2)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    ref = dgl.linear_cross_entropy(X, W, target, grad)
    assert all(torch.equal(x, y) for x, y in zip(ref, cap))


def test_two_streams_at_once():
    """Calls in flight on two streams share nothing but their inputs."""
    T, V, d = 900, 9001, 256
    X, W, target, grad = _inputs(T, V, d)
    ref = dgl.linear_cross_entropy(X, W, target, grad)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [dgl.linear_cross_entropy(X, W, target, grad, stream=s) for _ in range(4) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(x, y) for x, y in zip(ref, g))


def _teacher(T, V, k, seed=1, absent=0.2):
    g = _gen(seed)
    indices = torch.stack([torch.randperm(V, device=DEV, generator=g)[:k] for _ in range(T)]) if k <= V else \
        torch.randint(0, V, (T, k), device=DEV, generator=g)
    logits = 3.0 * torch.randn(T, k, device=DEV, generator=g)
    drop = torch.rand(T, k, device=DEV, generator=g) < absent
    indices = torch.where(drop, -1 - torch.randint(0, 5, (T, k), device=DEV, generator=g), indices)
    logits = torch.where(drop & (torch.rand(T, k, device=DEV, generator=g) < 0.5), float("nan"), logits)
    return indices.contiguous(), logits.float().contiguous()


@pytest.mark.parametrize("T,V,d,k", [(1, 1, 8, 1), (1, 300, 64, 1), (3, 129, 72, 5), (16, 11007, 128, 8),
                                     (129, 513, 264, 64), (200, 5000, 96, 128), (70, 131, 64, 128), (33, 50257, 64, 33)])
@pytest.mark.parametrize("temp", [1.0, 2.5])
def test_distill_sizes(T, V, d, k, temp):
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k)
    wanted = _wanted_distill(T, V, indices, logits, temp)
    for g in (None, grad):
        got = dgl.linear_distill(X, W, indices, logits, g, temperature=temp)
        _status()
        _check(X, W, 1.0 / temp, wanted, g, got)


def test_distill_rows_without_entries():
    T, V, d, k = 130, 600, 64, 6
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k)
    none = torch.zeros(T, dtype=torch.bool, device=DEV)
    none[[0, 64, 129]] = True
    indices[0] = -1
    indices[64] = -7
    logits[64] = float("nan")
    logits[129] = -float("inf")  # kept, but none has any probability
    indices[129] = torch.arange(k, device=DEV)
    X[none] = float("nan")
    got = dgl.linear_distill(X, W, indices, logits, grad)
    _status()
    assert (got[0][none] == 0).all() and (got[2][none] == 0).all()
    _check(X, W, 1.0, _wanted_distill(T, V, indices, logits, 1.0), grad, got, ignored_rows=none)
    indices.fill_(-1)
    got = dgl.linear_distill(X, W, indices, logits, grad)
    assert all((got[i] == 0).all() for i in (0, 2, 3))


def test_distill_extreme_logits():
    """Entries of minus infinity and of the type's lowest value weigh nothing; large ones do not overflow."""
    T, V, d, k = 40, 500, 64, 4
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k, absent=0.0)
    logits[:, 1] = -float("inf")
    logits[::2, 2] = torch.finfo(torch.float32).min
    logits[::3, 0] = 1e30
    got = dgl.linear_distill(X, W, indices, logits, grad)
    _status()
    wanted = _wanted_distill(T, V, indices, logits, 1.0)
    _check(X, W, 1.0, wanted[:3] + (100.0,), grad, got)


def test_distill_repeated_and_clustered_indices():
    T, V, d, k = 140, 400, 64, 12
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k, absent=0.1)
    indices[:, 3] = indices[:, 0]
    indices[:50, 7] = indices[:50, 0]
    indices[100:] = 5  # one token for all entries
    indices[60:80] = torch.arange(k, device=DEV) + 120  # neighbours, across a tile's edge
    logits = torch.nan_to_num(logits)
    got = dgl.linear_distill(X, W, indices, logits, grad)
    _status()
    _check(X, W, 1.0, _wanted_distill(T, V, indices, logits, 1.0), grad, got)


def test_distill_teacher_lse_keeps_the_tail_out():
    T, V, d, k = 100, 900, 64, 10
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k)
    clean = torch.where(indices >= 0, torch.nan_to_num(logits), -1e4)
    lse_t = torch.logsumexp(clean / 1.5, 1) + torch.rand(T, device=DEV, generator=_gen(4))
    lse_t = lse_t.float().contiguous()
    got = dgl.linear_distill(X, W, indices, logits, grad, temperature=1.5, teacher_lse=lse_t)
    _status()
    _check(X, W, 1.0 / 1.5, _wanted_distill(T, V, indices, logits, 1.5, lse_t), grad, got)


def test_distill_index_out_of_range():
    T, V, d, k = 60, 300, 64, 4
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k, absent=0.0)
    indices[8, 2] = V
    indices[9, 0] = 2**40
    got = dgl.linear_distill(X, W, indices, logits, grad)
    _status()
    assert got[0][8:10].isnan().all() and (got[2][8:10] == 0).all()
    indices[8:10] = -1
    loss = got[0].clone()
    loss[8:10] = 0
    _check(X, W, 1.0, _wanted_distill(T, V, indices, logits, 1.0), grad, (loss,) + got[1:])


def test_distill_wide_student_logits():
    T, V, d, k = 120, 2000, 64, 9
    X, W, _, grad = _inputs(T, V, d, w_std=0.01)
    W[:, 1] = torch.linspace(-1, 1, V, device=DEV).bfloat16()
    X[:, 1] = 200.0 * torch.linspace(-1, 1, T, device=DEV).bfloat16()
    indices, logits = _teacher(T, V, k)
    got = dgl.linear_distill(X, W, indices, logits, grad)
    _status()
    _check(X, W, 1.0, _wanted_distill(T, V, indices, logits, 1.0), grad, got)


def test_distill_of_one_entry_is_cross_entropy():
    T, V, d = 130, 700, 128
    X, W, target, grad = _inputs(T, V, d)
    a = dgl.linear_cross_entropy(X, W, target, grad)
    b = dgl.linear_distill(X, W, target[:, None].contiguous(), torch.zeros(T, 1, device=DEV), grad)
    _status()
    _check(X, W, 1.0, _wanted_xent(T, V, target), grad, b)
    assert torch.equal(a[1], b[1])


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_gradient_against_differences(op):
    """(L(X + D) - L(X - D)) / 2 along a direction D that bf16 holds exactly,
    against <dX, D>, and the same for W.  The central difference's own
    truncation is taken from the definition in 64 bits; the rest is the
    losses' rounding, 2^-18 |g| each, and dX's, 2^-7 of sum |dX D|."""
    T, V, d, k = 12, 300, 64, 5
    g = _gen(2)
    X = (torch.randint(-16, 17, (T, d), device=DEV, generator=g) / 16.0).bfloat16()
    W = (torch.randint(-16, 17, (V, d), device=DEV, generator=g) / 32.0).bfloat16()
    DX = (torch.randint(-1, 2, (T, d), device=DEV, generator=g) / 32.0).bfloat16()
    DW = (torch.randint(-1, 2, (V, d), device=DEV, generator=g) / 64.0).bfloat16()
    grad = torch.rand(T, device=DEV, generator=g)
    indices, logits = _teacher(T, V, k)
    target = torch.randint(0, V, (T,), device=DEV, generator=g)

    def own(x, w, up=None):
        if op == "xent":
            return dgl.linear_cross_entropy(x, w, target, up)
        return dgl.linear_distill(x, w, indices, logits, up)

    q, qlogq, live, _ = _wanted_xent(T, V, target) if op == "xent" else _wanted_distill(T, V, indices, logits, 1.0)

    def definition(x, w):
        z = x.double() @ w.double().T
        loss = qlogq - (q * z).sum(1) + q.sum(1) * torch.logsumexp(z, 1)
        return (grad.double() * torch.where(live, loss, 0.0)).sum().item()

    z = X.double() @ W.double().T
    dz = torch.where(live, grad.double(), 0.0)[:, None] * (q.sum(1, keepdim=True) * torch.softmax(z, 1) - q)
    _, _, dX, dW = own(X, W, grad)
    for ref, have, (xa, wa), (xb, wb), D in ((dz @ W.double(), dX, (X + DX, W), (X - DX, W), DX),
                                             (dz.T @ X.double(), dW, (X, W + DW), (X, W - DW), DW)):
        moved = 0.5 * ((own(xa, wa)[0].double() - own(xb, wb)[0].double()) * grad.double()).sum().item()
        along = (have.double() * D.double()).sum().item()
        cut = abs(0.5 * (definition(xa, wa) - definition(xb, wb)) - (ref * D.double()).sum().item())
        allowed = cut + T * 2.0**-18 + 2.0**-7 * (ref.abs() * D.double().abs()).sum().item()
        assert abs(moved - along) <= allowed, (moved, along, allowed)


def test_weights_past_2_31_elements():
    """Row offsets of W and dW that pass 32 bits."""
    T, V, d = 3, 270000, 8192
    g = _gen(0)
    X = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    W = torch.empty(V, d, device=DEV, dtype=torch.bfloat16).normal_(0, 0.01, generator=g)
    target = torch.tensor([V - 1, 5, V - 2], device=DEV)
    grad = torch.full((T,), 0.5, device=DEV)
    loss, lse, dX, dW = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    z = torch.cat([X.double() @ W[v:v + 30000].double().T for v in range(0, V, 30000)], 1)
    ref = torch.logsumexp(z, 1)
    ez = (d / 16 + 4) * 4 * 2.0**-24 * 0.01 * d
    assert (lse.double() - ref).abs().max() <= ez + 2.0**-20 * 20
    assert (loss.double() - (ref - z.gather(1, target[:, None])[:, 0])).abs().max() <= 2 * ez + 2.0**-20 * 40
    dz = 0.5 * torch.exp(z - ref[:, None])
    dz.scatter_add_(1, target[:, None], torch.full((T, 1), -0.5, dtype=torch.float64, device=DEV))
    for rows in (slice(0, 300), slice(V // 2, V // 2 + 300), slice(V - 300, V)):
        want = dz[:, rows].T @ X.double()
        tol = (3 * 2.0**-9 + 2.0**-8) * (dz[:, rows].abs().T @ X.double().abs())
        assert ((dW[rows].double() - want).abs() <= tol + 1e-12).all()
    want = sum(dz[:, v:v + 30000] @ W[v:v + 30000].double() for v in range(0, V, 30000))
    tol = sum(dz[:, v:v + 30000].abs() @ W[v:v + 30000].double().abs() for v in range(0, V, 30000))
    assert ((dX.double() - want).abs() <= (3 * 2.0**-9 + 2.0**-8) * tol).all()


def test_refusals_of_the_binding():
    X, W, target, grad = _inputs(10, 100, 64)
    with pytest.raises(TypeError):
        dgl.linear_cross_entropy(X.float(), W, target)
    with pytest.raises(TypeError):
        dgl.linear_cross_entropy(X, W, target.int())
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X, W[:, :32], target)
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X, W, target[:5])
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X, W, target, grad, need_dx=False, need_dw=False)
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X, W, target, grad, accumulate=True)
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X.T.contiguous().T, W, target)
    with pytest.raises(dgl.DglError):
        dgl.linear_cross_entropy(X, W, target, grad, dW=torch.empty(100, 64, device=DEV, dtype=torch.bfloat16),
                                 accumulate=True)
    with pytest.raises(dgl.DglError):  # d not a multiple of 8
        dgl.linear_cross_entropy(X[:, :60].contiguous(), W[:, :60].contiguous(), target)
    with pytest.raises(dgl.DglError):  # 2 bytes off a 16-byte boundary
        dgl.linear_cross_entropy(X[:, 1:57], W[:, :56], target)
    with pytest.raises(dgl.DglError):
        dgl.linear_cross_entropy(X, W, target, grad, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(dgl.DglError):
        dgl.linear_cross_entropy(X, W, target, logit_scale=float("nan"))
    with pytest.raises(ValueError):
        dgl.linear_distill(X, W, torch.zeros(10, 129, dtype=torch.int64, device=DEV), torch.zeros(10, 129, device=DEV))
    with pytest.raises(dgl.DglError):
        dgl.linear_distill(X, W, target[:, None].contiguous(), torch.zeros(10, 1, device=DEV), temperature=0.0)


def test_rows_that_overlap_are_refused():
    # one row seen as many has pitch 0, which the C call takes for packed rows: it would read past the buffer
    X, W, target, grad = _inputs(10, 100, 64)
    one = X[:1].expand(10, 64)
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(one, W, target)
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X, W[:1].expand(100, 64), target)
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X, W, target, grad, dW=torch.zeros(1, 64, device=DEV).expand(100, 64))
    with pytest.raises(ValueError):
        dgl.linear_distill(one, W, target[:, None].contiguous(), torch.zeros(10, 1, device=DEV))
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X.flatten().as_strided((10, 64), (8, 1)), W, target)
    # one token has no pitch
    loss, lse = dgl.linear_cross_entropy(X[:1].expand(1, 64), W, target[:1])
    z = X[:1].double() @ W.double().T
    assert torch.allclose(lse.double(), torch.logsumexp(z, 1), rtol=0, atol=1e-4)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, 7])
def test_dw_dtype_is_one_of_the_two(dtype):
    X, W, target, grad = _inputs(10, 100, 64)
    with pytest.raises(ValueError):
        dgl.linear_cross_entropy(X, W, target, grad, dw_dtype=dtype)
    assert dgl.linear_cross_entropy(X, W, target, grad, dw_dtype=dgl.OUT_F32)[3].dtype == torch.float32


def test_c_call_with_padded_rows_and_no_lse():
    """The C entry with a row pitch for every matrix, lse NULL and an fp32 dW: what lies between the rows stays."""
    T, V, d = 301, 777, 72
    X, W, target, grad = _inputs(T, V, d)
    want = dgl.linear_cross_entropy(X, W, target, grad, dw_dtype=dgl.OUT_F32)

    def padded(t, pad):
        p = torch.full((t.shape[0] + 1, t.shape[1] + pad), 5.0, device=DEV, dtype=t.dtype)
        p[:-1, :t.shape[1]] = t
        return p

    Xp, Wp = padded(X, 16), padded(W, 8)
    dXp, dWp = padded(torch.zeros_like(X), 24), padded(torch.zeros(V, d, device=DEV), 40)
    loss = torch.full((T + 1,), 5.0, device=DEV)
    h = dgl.HeadDesc(T=T, V=V, d=d, X=Xp.data_ptr(), ldx=d + 16, W=Wp.data_ptr(), ldw=d + 8, loss=loss.data_ptr(),
                     grad=grad.data_ptr(), dX=dXp.data_ptr(), lddx=d + 24, dW=dWp.data_ptr(), lddw=d + 40,
                     logit_scale=1.0, dw_dtype=dgl.OUT_F32)
    low, best = dgl.dgl_head_workspace(h)
    for size in (low, best):
        ws = torch.full((size + 256,), 255, dtype=torch.uint8, device=DEV)
        h.ws, h.ws_bytes = ws.data_ptr(), size
        assert dgl.dgl_linear_xent(h, target.data_ptr(), IGNORE, torch.cuda.current_stream().cuda_stream) == dgl.DGL_OK
        _status()
        assert (ws[size:] == 255).all()
        assert loss[T] == 5.0
        if size == best:  # the same chunks as the call above (chunks of 128 rows take other tiles)
            assert torch.equal(loss[:T], want[0]) and torch.equal(dXp[:T, :d], want[2])
            assert torch.equal(dWp[:V, :d], want[3])
        _check(X, W, 1.0, _wanted_xent(T, V, target), grad, (loss[:T], want[1], dXp[:T, :d], dWp[:V, :d]))
        for p, t in ((dXp, X), (dWp, W)):
            assert (p[-1] == 5.0).all() and (p[:, t.shape[1]:] == 5.0).all()


def test_distill_graph_in_chunks():
    T, V, d, k = 300, 1500, 64, 7
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k)
    low, _ = _workspace(T, V, d, k, dgl.OUT_BF16)
    ws = torch.empty(low, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap = dgl.linear_distill(X, W, indices, logits, grad, workspace=ws)
    X2, _, _, _ = _inputs(T, V, d, 8)
    X.copy_(X2)
    graph.replay()
    torch.cuda.synchronize()
    ref = dgl.linear_distill(X, W, indices, logits, grad, workspace=torch.empty_like(ws))
    _status()
    assert all(torch.equal(x, y) for x, y in zip(ref, cap))
    _check(X, W, 1.0, _wanted_distill(T, V, indices, logits, 1.0), grad, ref)
