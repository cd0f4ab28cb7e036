"""Rows that are nearly sure of their target: the loss and the target's dz are
what the other tokens leave, however large the target's logit is.

A hidden state has one element, so every logit is one exact product and the
tensor core rounds nothing.  With r = 1 - p the others' probability in 64 bits:

  each other token's term is off by its exponent's rounding, at most 2^-20
  (of about 15, in units of log 2) for the argument, 2^-22 for the
  exponential and 2^-24 of the logits' distance for the factor log2 e, and
  e's fp16 by 2^-12 of the term where a gradient's entry is formed from it:
  below 2^-17 r in a sum of them;
  adding them to the target's term rounds, a term at a time, by at most 2^-24
  of the sum; at most 48 additions meet the largest term (16 within a thread's
  share of a group, 3 of its shares, the row's groups and the reduction of a
  block's threads), and none of them rounds, or does anything, where the
  others together stay below 2^-26: then the loss is zero, and so is dz.

The sum takes in the target's own term, so no loss is below zero.
"""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from tests.test_gpu_head import DEV, _gen, _status

pytestmark = pytest.mark.gpu


def _sure(T, V, d, top, seed=0):
    """Rows whose largest logits reach from 1 to `top`, each the row's target; all products exact."""
    g = _gen(seed)
    W = (0.35 * torch.randn(V, d, device=DEV, generator=g)).bfloat16()
    rows = torch.arange(T, device=DEV)
    best, target = W[:, rows % d].max(0)  # [T]: the largest entry of each row's column
    # the second largest may be close by: half of the rows' targets stand apart
    apart = torch.rand(d, device=DEV, generator=g) < 0.5
    best = best[:d].float().abs()
    W[target[:d], rows[:d]] = torch.where(apart, 1.5 * best, best).bfloat16()
    size = top ** torch.rand(T, device=DEV, generator=g)
    X = torch.zeros(T, d, device=DEV)
    X[rows, rows % d] = size / W[target, rows % d].float()
    return X.bfloat16(), W, target


def _rest(X, W, target):
    z = X.double() @ W.double().T
    p = torch.softmax(z, 1)
    r = torch.where(torch.arange(W.shape[0], device=DEV) == target[:, None], 0.0, p).sum(1)
    return z, p, r


@pytest.mark.parametrize("top", [30.0, 200.0, 3000.0, 3.0e5])
@pytest.mark.parametrize("T,V", [(64, 9), (500, 300), (130, 7000)])
def test_loss_of_sure_rows(T, V, top):
    X, W, target = _sure(T, V, 64, top)
    z, p, r = _rest(X, W, target)
    want = -torch.log1p(-r)
    k = target[:, None].contiguous()
    for loss, lse in (dgl.linear_cross_entropy(X, W, target),
                      dgl.linear_distill(X, W, k, torch.zeros(T, 1, device=DEV))):
        _status()
        assert (loss >= 0).all(), f"{int((loss < 0).sum())} losses below zero, down to {loss.min().item():.3g}"
        off = (loss.double() - want).abs()
        tol = 2.0**-17 * want + torch.where(r < 2.0**-26, 2.0**-26, 48 * 2.0**-24)
        assert (off <= tol).all(), f"{int((off > tol).sum())} losses off, by up to {off[off > tol].max().item():.3g}"
        assert (loss[r < 2.0**-26] == 0).all()


@pytest.mark.parametrize("scale", [1.0, -1.0, 0.25])
def test_loss_of_sure_rows_scaled(scale):
    T, V = 300, 700
    X, W, target = _sure(T, V, 64, 200.0)
    X = (X.float() / scale).bfloat16()  # powers of two: exact
    _, _, r = _rest((X.float() * scale).bfloat16(), W, target)
    loss, _ = dgl.linear_cross_entropy(X, W, target, logit_scale=scale)
    _status()
    want = -torch.log1p(-r)
    assert (loss >= 0).all()
    assert ((loss.double() - want).abs() <= 2.0**-17 * want + torch.where(r < 2.0**-26, 2.0**-26, 48 * 2.0**-24)).all()


@pytest.mark.parametrize("top", [30.0, 200.0, 3000.0, 3.0e5])
@pytest.mark.parametrize("op", ["xent", "distill"])
def test_gradient_of_sure_rows(op, top):
    """dX = sum_v dz_v w_v: dz of the target is -r g to the bound above and 2^-8 of itself (bf16); the others'
    p g to 2^-8 of themselves, and nothing where they are below 2^-40 of their group's largest."""
    T, V, d = 500, 300, 64
    X, W, target = _sure(T, V, d, top)
    z, p, r = _rest(X, W, target)
    grad = torch.full((T,), 0.5, device=DEV)
    if op == "xent":
        _, _, dX, dW = dgl.linear_cross_entropy(X, W, target, grad, dw_dtype=dgl.OUT_F32)
    else:  # one certain entry and one of no weight
        k = torch.stack([target, (target + 1) % V], 1).contiguous()
        logits = torch.tensor([0.0, -200.0], device=DEV).repeat(T, 1).contiguous()
        _, _, dX, dW = dgl.linear_distill(X, W, k, logits, grad, dw_dtype=dgl.OUT_F32)
    _status()
    dz = 0.5 * p
    dz.scatter_(1, target[:, None], -0.5 * r[:, None])
    floor = torch.where(r < 2.0**-26, 2.0**-26, 48 * 2.0**-24).double()
    e_dz = (2.0**-8 + 2.0**-11) * dz.abs() + 0.5 * 2.0**-40
    e_dz.scatter_add_(1, target[:, None], 0.5 * floor[:, None])
    w, x = W.double(), X.double()
    for have, ref, err in ((dX, dz @ w, e_dz @ w.abs()), (dW, dz.T @ x, e_dz.T @ x.abs())):
        off = (have.double() - ref).abs()
        tol = err + 2.0**-8 * ref.abs() + 1e-30
        assert (off <= tol).all(), f"{int((off > tol).sum())} off, worst {(off / tol).max().item():.3g} of what is allowed"


def test_entries_of_little_weight_beside_a_sure_token():
    """A student sure of one token, whose teacher gives a thousandth to it and the rest to others: dz of each entry
    is Q p - w, to 2^-8 of itself."""
    T, V, d, k = 64, 300, 64, 4
    X, W, target = _sure(T, V, d, 60.0)
    _, p, _ = _rest(X, W, target)
    indices = torch.stack([(target + 7 * j) % V for j in range(k)], 1).contiguous()
    logits = torch.tensor([-7.0, 0.0, -1.0, -13.0], device=DEV).repeat(T, 1).contiguous()
    grad = torch.full((T,), 1.0, device=DEV)
    loss, _, dX, dW = dgl.linear_distill(X, W, indices, logits, grad, dw_dtype=dgl.OUT_F32)
    _status()
    q = torch.zeros_like(p).scatter_add_(1, indices, torch.softmax(logits.double(), 1))
    dz = p - q
    e_dz = (2.0**-8 + 2.0**-11) * dz.abs() + 2.0**-17 * p + 48 * 2.0**-24 * (p > 0.25) + 2.0**-20 * q + 2.0**-40
    w, x = W.double(), X.double()
    for have, ref, err in ((dX, dz @ w, e_dz @ w.abs()), (dW, dz.T @ x, e_dz.T @ x.abs())):
        assert ((have.double() - ref).abs() <= err + 2.0**-8 * ref.abs() + 1e-30).all()
