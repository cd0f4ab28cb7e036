"""linear_distill's teacher distribution at logits whose size hides their differences.

Softmax does not change when one number is added to all logits of a row, so
its weights follow the entries' differences however large the entries are.
Tolerances are test_gpu_head's: none of them grows with the teacher's logits
(a difference of two nearby fp32 numbers is exact)."""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from tests.test_gpu_head import DEV, _check, _gen, _inputs, _status, _wanted_distill

pytestmark = pytest.mark.gpu


def _near(T, V, k, level, step, seed=5):
    """Entries `level` - step n, n small whole numbers, two or more of them at the level itself."""
    g = _gen(seed)
    indices = torch.stack([torch.randperm(V, device=DEV, generator=g)[:k] for _ in range(T)])
    n = torch.randint(0, 4, (T, k), device=DEV, generator=g)
    n[:, :2] = 0
    return indices.contiguous(), (level - step * n).float().contiguous()


def _wanted(T, V, indices, logits, temp):
    """The definition at the logits less their largest, exact in fp32 here: even 64 bits do not hold log 3 beside 3e38."""
    q, qlogq, live, big = _wanted_distill(T, V, indices, logits - logits.amax(1, keepdim=True), temp)
    return q, qlogq, live, min(big, 100.0)  # an entry without weight has no part in the loss's rounding


@pytest.mark.parametrize("k", [3, 40, 128])
@pytest.mark.parametrize("level,step", [(1e4, 0.5), (1e8, 8.0), (-1e5, 0.25), (3e38, 2.0**104)])
def test_distill_large_teacher_logits(level, step, k):
    T, V, d = 70, 500, 64
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _near(T, V, k, level, step)
    got = dgl.linear_distill(X, W, indices, logits, grad)
    _status()
    _check(X, W, 1.0, _wanted(T, V, indices, logits, 1.0), grad, got)


@pytest.mark.parametrize("temp", [0.7, 1.5, 4.0])
def test_distill_large_teacher_logits_at_a_temperature(temp):
    """The temperature divides the differences, not the logits: each quotient's own rounding would be as large as
    the differences of its neighbours."""
    T, V, d, k = 70, 500, 64, 9
    X, W, _, grad = _inputs(T, V, d)
    for level, step in ((1e5, 0.25), (1e8, 8.0)):
        indices, logits = _near(T, V, k, level, step)
        got = dgl.linear_distill(X, W, indices, logits, grad, temperature=temp)
        _status()
        _check(X, W, 1.0 / temp, _wanted(T, V, indices, logits, temp), grad, got)


def test_distill_weights_sum_to_one_at_any_size():
    """With a student that is uniform (W = 0) a row's loss is sum q log q + Q log V: log V - log 3 for three equal
    entries, to 2^-20 of the terms, and its dX is zero."""
    T, V, d = 40, 300, 64
    X, _, _, grad = _inputs(T, V, d)
    W = torch.zeros(V, d, device=DEV, dtype=torch.bfloat16)
    indices = torch.arange(3, device=DEV).repeat(T, 1).contiguous()
    logits = (10.0 ** torch.linspace(0, 38, T, device=DEV, dtype=torch.float64)).float()[:, None].repeat(1, 3).contiguous()
    logits[::2] *= -1
    loss, lse, dX, _ = dgl.linear_distill(X, W, indices, logits, grad)
    _status()
    want = torch.tensor(V / 3.0, dtype=torch.float64).log().item()
    assert (loss.double() - want).abs().max() <= 2.0**-20 * 10
    assert (dX == 0).all()
