"""The common significand of the rows' grad stays out of dz's rounding, whichever
rows of the call carry it.

grad = 1 + 2^-8 in every row lies half-way between two bf16 numbers, so dz = -grad
rounds by 2^-8 of itself where it is formed whole.  Students that are nearly
uniform (p about 1 / V) leave of dW = dz^T x little but the targets' entries:
rounded whole, dW is off by 2^-8 (0.0039) of its norm; without the grad's
significand a target's entry is -(1 - p) times a power of two, off by at most
p + 2^-24, and the others by 2^-8 p.  dX is rounded to bf16 itself, 2^-8 at most
and 2^-8 / sqrt(3) in the mean square over many entries.
"""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from tests.test_gpu_head import DEV, IGNORE, _gen, _status

pytestmark = pytest.mark.gpu

GRAD = 1.0 + 2.0**-8


@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("zeros,how", [(0, "grad"), (31, "grad"), (40, "grad"), (300, "grad"), (1100, "grad"), (700, "ignored")])
@pytest.mark.parametrize("workspace", ["one chunk", "chunks"])
def test_common_significand(op, zeros, how, workspace):
    _common_significand(op, zeros, how, workspace, 8192)


def test_common_significand_of_long_rows():
    """Rows past 32768 columns, each finished by one larger block."""
    _common_significand("xent", 1100, "grad", "one chunk", 40001)


def _common_significand(op, zeros, how, workspace, V):
    T, d = zeros + 150, 64
    g = _gen(0)
    X = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    W = (0.002 * torch.randn(V, d, device=DEV, generator=g)).bfloat16()
    target = torch.randperm(V, device=DEV, generator=g)[:T].contiguous()
    grad = torch.full((T,), GRAD, device=DEV)
    grad[:zeros] = 0.0
    if how == "ignored":
        target[:zeros] = IGNORE
    ws = None
    if workspace == "chunks":
        h = dgl.HeadDesc(T=T, V=V, d=d, grad=1, dX=1, dW=1, dw_dtype=dgl.OUT_F32)
        ws = torch.empty(dgl.dgl_head_workspace(h, 0 if op == "xent" else 1)[0], dtype=torch.uint8, device=DEV)
    if op == "xent":
        _, _, dX, dW = dgl.linear_cross_entropy(X, W, target, grad, dw_dtype=dgl.OUT_F32, workspace=ws)
    else:
        _, _, dX, dW = dgl.linear_distill(X, W, target[:, None].contiguous(), torch.zeros(T, 1, device=DEV), grad,
                                          dw_dtype=dgl.OUT_F32, workspace=ws)
    _status()
    x, w = X.double(), W.double()
    p = torch.softmax(x @ w.T, 1)
    dz = p.clone()
    at = target.clamp(min=0)[:, None]
    dz.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0))
    dz *= grad.double()[:, None]
    want = dz.T @ x
    e_dz = 2.0**-8 * dz.abs()
    e_dz.scatter_(1, at, (p.gather(1, at) + 2.0**-20) * grad.double()[:, None])
    bound = ((e_dz.T @ x.abs()).norm() / want.norm()).item()
    assert bound < 0.5 * 2.0**-8, "the inputs do not tell the two apart"
    off = ((dW.double() - want).norm() / want.norm()).item()
    assert off <= bound, f"dW is off by {off:.2e} of its norm, {bound:.2e} is allowed"
    want = dz @ w
    off = ((dX.double() - want).norm() / want.norm()).item()
    # (dX's other entries of dz average out: below a tenth of the rounding)
    assert off <= 1.1 * 2.0**-8 / 3**0.5, f"dX is off by {off:.2e} of its norm"


def test_no_grad_at_all():
    """A grad of nothing but zeros: no gradient, and no NaN."""
    T, V, d = 300, 500, 64
    g = _gen(1)
    X = torch.randn(T, d, device=DEV, generator=g).bfloat16()
    W = torch.randn(V, d, device=DEV, generator=g).bfloat16()
    target = torch.randint(0, V, (T,), device=DEV, generator=g)
    loss, _, dX, dW = dgl.linear_cross_entropy(X, W, target, torch.zeros(T, device=DEV))
    _status()
    assert not loss.isnan().any() and (dX == 0).all() and (dW == 0).all()
