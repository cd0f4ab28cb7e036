"""One gradient of a head alone (a frozen head has no dW) within the scratch that is
reported for it, in one chunk and in chunks; the same bits as with both."""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from tests.test_gpu_head import DEV, IGNORE, _check, _inputs, _status, _teacher, _wanted_distill, _wanted_xent

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("need", [(True, False), (False, True)], ids=["dX", "dW"])
@pytest.mark.parametrize("op", ["xent", "distill"])
@pytest.mark.parametrize("T,V,d", [(1, 300, 64), (140, 1000, 72), (1000, 5003, 256)])
def test_one_gradient_within_its_workspace(T, V, d, op, need):
    X, W, target, grad = _inputs(T, V, d)
    target[::5] = IGNORE
    X[::5] = float("nan")  # rows without a target, in neither gradient
    k = 0 if op == "xent" else 6
    if k:
        indices, logits = _teacher(T, V, k)
        indices[::5] = -1
    ignored = torch.zeros(T, dtype=torch.bool, device=DEV)
    ignored[::5] = True

    def call(**kw):
        if op == "xent":
            return dgl.linear_cross_entropy(X, W, target, grad, dw_dtype=dgl.OUT_F32, **kw)
        return dgl.linear_distill(X, W, indices, logits, grad, dw_dtype=dgl.OUT_F32, **kw)

    wanted = _wanted_xent(T, V, target) if op == "xent" else _wanted_distill(T, V, indices, logits, 1.0)
    both = call()
    h = dgl.HeadDesc(T=T, V=V, d=d, grad=1, dX=need[0], dW=need[1], dw_dtype=dgl.OUT_F32)
    low, best = dgl.dgl_head_workspace(h, k)
    for size in (low, best):
        buf = torch.full((size + 256,), 255, dtype=torch.uint8, device=DEV)  # NaN whatever type is read
        got = call(need_dx=need[0], need_dw=need[1], workspace=buf[:size])
        _status()
        assert (buf[size:] == 255).all(), "wrote past the workspace"
        assert [g is None for g in got[2:]] == [not n for n in need]
        _check(X, W, 1.0, wanted, grad, got, ignored_rows=ignored)
        if size == best:
            assert all(torch.equal(a, b) for a, b in zip(got[2:], both[2:]) if a is not None)
            assert torch.equal(got[0], both[0])
