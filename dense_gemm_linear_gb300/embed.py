"""Embedding lookup and its gradient on torch CUDA tensors (dgl_embedding, dgl_embedding_grad).

The helpers check their arguments, allocate what is not passed in with torch,
and make one call of the library on torch's current stream.  The tensors are on
the current device, where the library launches.
"""
from __future__ import annotations

import functools

import torch

from . import OUT_BF16, OUT_F32, EmbedDesc, _check, dgl_embedding_workspace, load_library
from .head import _byref, _not_here, _on_stream, _packed, _rows
from .norm import _matrix

_TYPES = {OUT_BF16: torch.bfloat16, OUT_F32: torch.float32}


def _count(tokens):
    if not isinstance(tokens, torch.Tensor) or tokens.dim() != 1:
        raise TypeError("tokens must be a 1-D int64 CUDA tensor")
    return tokens.shape[0]


@functools.lru_cache(maxsize=256)
def _workspace_bytes(T, V, d, w_dtype, y_dtype):
    return dgl_embedding_workspace(EmbedDesc(T=T, V=V, d=d, w_dtype=w_dtype, y_dtype=y_dtype))


def embedding(tokens, W, *, scale=1.0, ignore_index=-100, out_dtype=None, out=None, stream=None):
    """Y[t] = scale W[tokens[t]]: a row of W for each token.

    tokens int64 [T], W [V, d] bf16 or fp32 (rows may be strided).  Returns Y
    [T, d] of out_dtype (OUT_BF16 or OUT_F32; W's type when None), or `out`.  A token
    equal to ignore_index gives zeros, any other outside [0, V) NaN.  All
    tensors are on the current device (stream's, when one is given).
    """
    if stream is not None:
        return _on_stream(stream, lambda: embedding(tokens, W, scale=scale, ignore_index=ignore_index,
                                                    out_dtype=out_dtype, out=out), tokens, W, out)
    T = _count(tokens)
    w_code, V, d = _matrix(W, "W")
    device = torch.cuda.current_device()
    at = _packed(tokens, "tokens", torch.int64, (T,), device)
    ldw = _rows(W, "W", W.dtype, (V, d), device)
    if out is None:
        y_code = w_code if out_dtype is None else out_dtype
        if y_code not in _TYPES:
            raise ValueError("out_dtype must be OUT_BF16 or OUT_F32")
        out = torch.empty((T, d), dtype=_TYPES[y_code], device=device)
        ldy = d
    else:
        y_code = _matrix(out, "out")[0]
        if out_dtype is not None and out_dtype != y_code:
            raise TypeError("out is not of out_dtype")
        ldy = _rows(out, "out", out.dtype, (T, d), device)
    e = EmbedDesc(T, V, d, at, ignore_index, W.data_ptr(), None, ldw, out.data_ptr(), None, ldy, scale=scale,
                  w_dtype=w_code, y_dtype=y_code)
    st = load_library().dgl_embedding(_byref(e), torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_embedding")
    return out


def embedding_grad(tokens, dY, V, *, scale=1.0, ignore_index=-100, dW=None, dw_dtype=OUT_BF16, accumulate=False,
                   workspace=None, stream=None):
    """dW[v] = scale times the sum of dY's rows whose token is v.

    tokens int64 [T], dY [T, d] bf16 or fp32 (rows may be strided), V the
    vocabulary.  Returns dW [V, d], bf16 or fp32 (dw_dtype, or the type of the dW passed in).
    accumulate adds to an fp32 dW, such as the one that the loss of a head
    with the same weights left.  Tokens equal to ignore_index or outside [0, V) add
    nothing.  workspace: a CUDA buffer of at least dgl_embedding_workspace
    bytes, made when None.
    """
    if stream is not None:
        return _on_stream(stream, lambda: embedding_grad(
            tokens, dY, V, scale=scale, ignore_index=ignore_index, dW=dW, dw_dtype=dw_dtype, accumulate=accumulate,
            workspace=workspace), tokens, dY, dW, workspace)
    T = _count(tokens)
    y_code, _, d = _matrix(dY, "dY")
    device = torch.cuda.current_device()
    at = _packed(tokens, "tokens", torch.int64, (T,), device)
    ldy = _rows(dY, "dY", dY.dtype, (T, d), device)
    if dw_dtype not in _TYPES:
        raise ValueError("dw_dtype must be OUT_BF16 or OUT_F32")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate adds to the fp32 dW that is passed in")
        dW = torch.empty((V, d), dtype=_TYPES[dw_dtype], device=device)
        ldw = d
    else:
        dw_dtype = _matrix(dW, "dW")[0]
        ldw = _rows(dW, "dW", dW.dtype, (V, d), device)
    if workspace is None:
        workspace = torch.empty(max(1, _workspace_bytes(T, V, d, dw_dtype, y_code)), dtype=torch.uint8, device=device)
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != device:
            _not_here(workspace, "workspace", device)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor")
    e = EmbedDesc(T, V, d, at, ignore_index, None, dW.data_ptr(), ldw, None, dY.data_ptr(), ldy, workspace.data_ptr(),
                  workspace.nbytes, scale, dw_dtype, y_code, 1 if accumulate else 0)
    st = load_library().dgl_embedding_grad(_byref(e), torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_embedding_grad")
    return dW
