"""Embedding lookup and its gradient on torch CUDA tensors (dgl_embedding, dgl_embedding_grad).

The helpers check their arguments, allocate what is not passed in with torch,
and make one call of the library on torch's current stream.  The tensors are on
the current device, where the library launches.  What a call checks of its tensors'
types, extents and strides is kept for the next call with the same.
"""
from __future__ import annotations

import functools

import torch

from . import OUT_BF16, EmbedDesc, _check, _packer, dgl_embedding_workspace, load_library
from .head import _on_stream
from .norm import _TYPES, _buffer, _matrix, _meta, _vector

_pack = _packer(EmbedDesc)


def _count(tokens, device):
    if tokens is None or len(tokens[2]) != 1:
        raise TypeError("tokens must be a 1-D int64 CUDA tensor")
    _vector(tokens, "tokens", device, tokens[2][0], torch.int64)
    return tokens[2][0]


@functools.lru_cache(maxsize=1024)
def _lookup(device, tokens, W, out_dtype, out):
    w_code, ldw = _matrix(W, "W", device)
    T, d = _count(tokens, device), W[2][1]
    if out is None:
        y_code = w_code if out_dtype is None else out_dtype
        if y_code not in _TYPES:
            raise ValueError("out_dtype must be OUT_BF16 or OUT_F32")
        return w_code, ldw, y_code, d
    y_code, ldy = _matrix(out, "out", device, (T, d))
    if out_dtype is not None and out_dtype != y_code:
        raise TypeError("out is not of out_dtype")
    return w_code, ldw, y_code, ldy


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
    device = torch.cuda.current_device()
    w_code, ldw, y_code, ldy = _lookup(device, _meta(tokens), _meta(W), out_dtype, _meta(out))
    (T,), (V, d) = tokens.shape, W.shape
    if out is None:
        out = torch.empty((T, d), dtype=_TYPES[y_code], device=device)
    e = _pack(T, V, d, tokens.data_ptr(), ignore_index, W.data_ptr(), 0, ldw, out.data_ptr(), 0, ldy, 0, 0, scale, w_code,
              y_code, 0)
    st = load_library().dgl_embedding(e, torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_embedding")
    return out


@functools.lru_cache(maxsize=1024)
def _gradient(device, tokens, dY, V, dW, dw_dtype, accumulate):
    y_code, ldy = _matrix(dY, "dY", device)
    T, d = _count(tokens, device), dY[2][1]
    if dY[2][0] != T:
        raise ValueError(f"dY must have shape {(T, d)}")
    if dw_dtype not in _TYPES:
        raise ValueError("dw_dtype must be OUT_BF16 or OUT_F32")
    if dW is None:
        if accumulate:
            raise ValueError("accumulate adds to the fp32 dW that is passed in")
        ldw = d
    else:
        dw_dtype, ldw = _matrix(dW, "dW", device, (V, d))
    size = dgl_embedding_workspace(EmbedDesc(T=T, V=V, d=d, w_dtype=dw_dtype, y_dtype=y_code))
    return y_code, ldy, dw_dtype, ldw, max(1, size)


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
    device = torch.cuda.current_device()
    y_code, ldy, dw_dtype, ldw, size = _gradient(device, _meta(tokens), _meta(dY), V, _meta(dW), dw_dtype, accumulate)
    T, d = dY.shape
    if dW is None:
        dW = torch.empty((V, d), dtype=_TYPES[dw_dtype], device=device)
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=device)
    else:
        _buffer(workspace, device)
        size = workspace.nbytes
    e = _pack(T, V, d, tokens.data_ptr(), ignore_index, 0, dW.data_ptr(), ldw, 0, dY.data_ptr(), ldy, workspace.data_ptr(),
              size, scale, dw_dtype, y_code, 1 if accumulate else 0)
    st = load_library().dgl_embedding_grad(e, torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_embedding_grad")
    return dW
