"""The head losses' arguments in the combinations that training uses: a logit scale
with a temperature, distillation that adds to a main gradient in chunks, 128
entries with the teacher's normaliser, wide hidden states, large vocabularies."""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from tests.test_gpu_head import DEV, _check, _gen, _inputs, _status, _teacher, _wanted_distill, _wanted_xent

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.25, -0.7, 3.0])
@pytest.mark.parametrize("temp", [0.8, 2.0])
def test_distill_logit_scale_with_temperature(scale, temp):
    """The scale is the student's alone; the temperature divides both sides."""
    T, V, d, k = 150, 900, 64, 7
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k)
    got = dgl.linear_distill(X, W, indices, logits, grad, temperature=temp, logit_scale=scale)
    _status()
    _check(X, W, scale / temp, _wanted_distill(T, V, indices, logits, temp), grad, got)


@pytest.mark.parametrize("T", [90, 300])
@pytest.mark.parametrize("small", [False, True], ids=["one chunk", "chunks"])
def test_distill_accumulates(T, small):
    V, d, k = 650, 80, 5
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k)
    before = torch.randn(V, d, device=DEV, generator=_gen(9)) * 0.05
    h = dgl.HeadDesc(T=T, V=V, d=d, grad=1, dX=1, dW=1, dw_dtype=dgl.OUT_F32)
    ws = torch.empty(dgl.dgl_head_workspace(h, k)[0], dtype=torch.uint8, device=DEV) if small else None
    dW = before.clone()
    got = dgl.linear_distill(X, W, indices, logits, grad, dW=dW, accumulate=True, workspace=ws)
    _status()
    assert got[3] is dW
    _check(X, W, 1.0, _wanted_distill(T, V, indices, logits, 1.0), grad, got, dw_before=before)


def test_distill_128_entries_with_the_teachers_normaliser():
    T, V, d, k = 200, 3000, 96, 128
    X, W, _, grad = _inputs(T, V, d)
    indices, logits = _teacher(T, V, k)
    clean = torch.where(indices >= 0, torch.nan_to_num(logits), -1e4)
    lse = (torch.logsumexp(clean / 1.5, 1) + torch.rand(T, device=DEV, generator=_gen(4))).float().contiguous()
    got = dgl.linear_distill(X, W, indices, logits, grad, temperature=1.5, teacher_lse=lse)
    _status()
    _check(X, W, 1.0 / 1.5, _wanted_distill(T, V, indices, logits, 1.5, lse), grad, got)


@pytest.mark.parametrize("T,V,d", [(40, 300, 8200), (3, 140001, 64), (150, 140001, 72)])
def test_wide_states_and_large_vocabularies(T, V, d):
    X, W, target, grad = _inputs(T, V, d, w_std=0.02)
    got = dgl.linear_cross_entropy(X, W, target, grad)
    _status()
    _check(X, W, 1.0, _wanted_xent(T, V, target), grad, got)
