"""Losses of a linear head on torch CUDA tensors (dgl_linear_xent, dgl_linear_distill).

The helpers check their arguments, allocate what is not passed in with torch,
and make one call of the library on torch's current stream.  The tensors are on
the current device, where the library launches.  On a few tokens
the kernels take about as long as this module does, so the checks are written
out rather than shared.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import DISTILL_MAX_K, OUT_BF16, OUT_F32, HeadDesc, _check, dgl_head_workspace, load_library

_BF16, _F32, _I64 = torch.bfloat16, torch.float32, torch.int64
_byref = ctypes.byref


def _not_here(t, name, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    raise ValueError(f"{name} is on cuda:{t.get_device()}, but the current device is cuda:{device}")


def _rows(t, name, dtype, shape, device):
    """Checks a matrix of `shape` whose rows are contiguous on the current device, where the library launches;
    returns its row pitch in elements."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _not_here(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    pitch, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if shape[0] <= 1:
        return shape[1]
    if pitch < shape[1]:  # a row repeated by expand() has pitch 0, which the C call reads as packed rows
        raise ValueError(f"the rows of {name} must not overlap")
    return pitch


def _packed(t, name, dtype, shape, device):
    """Checks a contiguous tensor on the current device; returns its address."""
    if not isinstance(t, torch.Tensor) or t.get_device() != device:
        _not_here(t, name, device)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}")
    return t.data_ptr()


@functools.lru_cache(maxsize=256)
def _workspace_bytes(T, V, d, grad, dX, dW, dw_dtype, k):
    h = HeadDesc(T=T, V=V, d=d, grad=grad, dX=dX, dW=dW, dw_dtype=dw_dtype)
    return max(1, dgl_head_workspace(h, k)[1])


def _head(X, W, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace, k, device):
    """Checks and allocates on the current stream; returns the descriptor and the tensors to return."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2 or not isinstance(W, torch.Tensor) or W.dim() != 2:
        raise TypeError("X and W must be 2-D CUDA tensors")
    T, d = X.shape
    V = W.shape[0]
    ldx = _rows(X, "X", _BF16, (T, d), device)
    ldw = _rows(W, "W", _BF16, (V, d), device)
    if dw_dtype not in (OUT_BF16, OUT_F32):
        raise ValueError("dw_dtype must be OUT_BF16 or OUT_F32")
    p_grad = p_dx = p_dw = lddw = 0
    dw_type = OUT_BF16
    dX = None
    if grad is not None:
        p_grad = _packed(grad, "grad", _F32, (T,), device)
        if not (need_dx or need_dw):
            raise ValueError("a call with grad computes dX, dW or both")
        if need_dx:
            dX = torch.empty((T, d), dtype=_BF16, device=device)
            p_dx = dX.data_ptr()
        if need_dw:
            if dW is None:
                if accumulate:
                    raise ValueError("accumulate adds to the fp32 dW that is passed in")
                dw_type = dw_dtype
                dW = torch.empty((V, d), dtype=_F32 if dw_type == OUT_F32 else _BF16, device=device)
                lddw = d
            else:
                if dW.dtype not in (_F32, _BF16):
                    raise TypeError(f"dW must be fp32 or bf16, got {dW.dtype}")
                lddw = _rows(dW, "dW", dW.dtype, (V, d), device)
                dw_type = OUT_F32 if dW.dtype == _F32 else OUT_BF16
            p_dw = dW.data_ptr()
        elif dW is not None or accumulate:
            raise ValueError("dW is given but not asked for")
    elif dW is not None or accumulate:
        raise ValueError("dW needs grad, the losses' upstream gradient")
    loss = torch.empty(T, dtype=_F32, device=device)
    lse = torch.empty(T, dtype=_F32, device=device)
    if workspace is None:
        size = _workspace_bytes(T, V, d, p_grad != 0, p_dx != 0, p_dw != 0, dw_type, k)
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != device:
            _not_here(workspace, "workspace", device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
    h = HeadDesc(T, V, d, X.data_ptr(), ldx, W.data_ptr(), ldw, loss.data_ptr(), lse.data_ptr(), p_grad, p_dx, d, p_dw,
                 lddw, workspace.data_ptr(), workspace.nbytes, logit_scale, dw_type, 1 if accumulate else 0)
    # the workspace is returned to be held until the call has been made
    return h, ((loss, lse) if grad is None else (loss, lse, dX, dW)), workspace


def _on_stream(stream, call, *tensors):
    """Makes a call on `stream` in place of the current one."""
    # buffers made by the call belong to the stream that uses them, and the
    # caller's are marked as used there: the allocator hands either out again
    # only after its work
    with torch.cuda.stream(stream):
        out = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return out


def linear_cross_entropy(X, W, target, grad=None, *, ignore_index=-100, logit_scale=1.0, need_dx=True, need_dw=True,
                         dW=None, dw_dtype=OUT_BF16, accumulate=False, workspace=None, stream=None):
    """Softmax cross entropy of the head z = logit_scale X . W^T, without keeping the logits.

    X [T, d], W [V, d] bf16 (rows may be strided), target int64 [T].  Returns
    (loss, lse), fp32 [T] each.  With grad, fp32 [T], the gradient of the
    final scalar by each loss (1 / tokens for a mean), returns (loss, lse, dX,
    dW): dX bf16, dW bf16 or fp32 (dw_dtype, or the type of the dW passed in;
    accumulate adds to an fp32 dW).  workspace: a CUDA buffer of at least
    dgl_head_workspace bytes, made when None.  All tensors are on the current
    device (stream's, when one is given).
    """
    if stream is not None:
        return _on_stream(stream, lambda: linear_cross_entropy(
            X, W, target, grad, ignore_index=ignore_index, logit_scale=logit_scale, need_dx=need_dx, need_dw=need_dw,
            dW=dW, dw_dtype=dw_dtype, accumulate=accumulate, workspace=workspace), X, W, target, grad, dW, workspace)
    device = torch.cuda.current_device()
    h, out, held = _head(X, W, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace, 0, device)
    at = _packed(target, "target", _I64, (X.shape[0],), device)
    st = load_library().dgl_linear_xent(_byref(h), at, ignore_index, torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_linear_xent")
    return out


def linear_distill(X, W, indices, logits, grad=None, *, temperature=1.0, teacher_lse=None, logit_scale=1.0,
                   need_dx=True, need_dw=True, dW=None, dw_dtype=OUT_BF16, accumulate=False, workspace=None,
                   stream=None):
    """Distillation of the head z = logit_scale X . W^T from a teacher's top logits.

    indices int64 [T, k] (negative: absent) and logits fp32 [T, k] are the
    teacher's; loss_t is the Kullback-Leibler divergence of the student's
    softmax(z / temperature) from the teacher's distribution over the entries
    (with teacher_lse, fp32 [T], from its share of the whole vocabulary's).
    Otherwise as linear_cross_entropy.
    """
    if stream is not None:
        return _on_stream(stream, lambda: linear_distill(
            X, W, indices, logits, grad, temperature=temperature, teacher_lse=teacher_lse, logit_scale=logit_scale,
            need_dx=need_dx, need_dw=need_dw, dW=dW, dw_dtype=dw_dtype, accumulate=accumulate, workspace=workspace),
            X, W, indices, logits, grad, teacher_lse, dW, workspace)
    k = indices.shape[1] if indices.dim() == 2 else 0
    if not 1 <= k <= DISTILL_MAX_K:
        raise ValueError(f"indices must be [T, k] with 1 <= k <= {DISTILL_MAX_K}")
    device = torch.cuda.current_device()
    h, out, held = _head(X, W, grad, logit_scale, need_dx, need_dw, dW, dw_dtype, accumulate, workspace, k, device)
    shape = (X.shape[0], k)
    at = _packed(indices, "indices", _I64, shape, device)
    values = _packed(logits, "logits", _F32, shape, device)
    lse_at = None if teacher_lse is None else _packed(teacher_lse, "teacher_lse", _F32, shape[:1], device)
    st = load_library().dgl_linear_distill(_byref(h), at, values, lse_at, k, temperature,
                                           torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_linear_distill")
    return out
