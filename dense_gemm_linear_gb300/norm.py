"""Layer norm on torch CUDA tensors (dgl_layer_norm, dgl_layer_norm_grad).

The helpers check their arguments, allocate what is not passed in with torch,
and make one call of the library on torch's current stream.  The tensors are on
the current device, where the library launches.  On a few rows the kernels take
less time than this module does, so what a call checks of its tensors' types,
extents and strides is kept for the next call with the same.
"""
from __future__ import annotations

import functools

import torch

from . import OUT_BF16, OUT_F32, NormDesc, _check, _packer, dgl_layer_norm_workspace, load_library
from .head import _on_stream

_F32 = torch.float32
_pack = _packer(NormDesc)
_CODES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}
_TYPES = {OUT_BF16: torch.bfloat16, OUT_F32: torch.float32}


def _meta(t):
    """What is checked of a tensor (None: not given)."""
    if t is None:
        return None
    try:
        return t.get_device(), t.dtype, t.shape, t.stride()
    except AttributeError:
        raise TypeError(f"a CUDA tensor is expected, got {type(t).__name__}") from None


def _here(meta, name, device):
    if meta is None or meta[0] < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if meta[0] != device:
        raise ValueError(f"{name} is on cuda:{meta[0]}, but the current device is cuda:{device}")


def _type(meta, name):
    code = _CODES.get(meta[1])
    if code is None:
        raise TypeError(f"{name} must be bf16 or fp32, got {meta[1]}")
    return code


def _matrix(meta, name, device, shape=None, dtype=None):
    """Checks a matrix whose rows are contiguous; returns its type code and row pitch in elements."""
    _here(meta, name, device)
    code = _type(meta, name)
    if dtype is not None and meta[1] != dtype:
        raise TypeError(f"{name} must be {dtype}, got {meta[1]}")
    if len(meta[2]) != 2 or (shape is not None and meta[2] != shape):
        raise ValueError(f"{name} must have " + ("two dimensions" if shape is None else f"shape {tuple(shape)}"))
    (rows, cols), (pitch, step) = meta[2], meta[3]
    if step != 1 and cols > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if rows <= 1:
        return code, cols
    if pitch < cols:  # a row repeated by expand() has pitch 0, which the C call reads as packed rows
        raise ValueError(f"the rows of {name} must not overlap")
    return code, pitch


def _vector(meta, name, device, length, dtype):
    """Checks a contiguous vector."""
    _here(meta, name, device)
    if meta[1] != dtype:
        raise TypeError(f"{name} must be {dtype}, got {meta[1]}")
    if tuple(meta[2]) != (length,) or (length > 1 and meta[3] != (1,)):
        raise ValueError(f"{name} must be a contiguous tensor of shape {(length,)}")


def _buffer(workspace, device):
    """Checks a scratch buffer."""
    meta = _meta(workspace)
    _here(meta, "workspace", device)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")


def _columns(device, d, weight, bias):
    """The type code of the weight and the bias."""
    code = OUT_F32
    for meta, name in ((weight, "weight"), (bias, "bias")):
        if meta is None:
            continue
        _here(meta, name, device)
        code = _type(meta, name)
        _vector(meta, name, device, d, meta[1])
    if weight is not None and bias is not None and weight[1] != bias[1]:
        raise TypeError("weight and bias must have the same type")
    return code


@functools.lru_cache(maxsize=1024)
def _forward(device, x, weight, bias, out):
    code, ldx = _matrix(x, "x", device)
    w_code = _columns(device, x[2][1], weight, bias)
    ldy = x[2][1] if out is None else _matrix(out, "out", device, x[2], x[1])[1]
    return code, ldx, w_code, ldy


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, out=None, stream=None):
    """y = (x - mean) rstd weight + bias over the rows of x, with the statistics that the gradient reads.

    x [rows, d] bf16 or fp32 (rows may be strided); weight and bias [d], bf16 or
    fp32, or None.  Returns (y, mean, rstd): y of x's type (or `out`, which may be x),
    mean and rstd fp32 [rows].  All tensors are on the current device (stream's,
    when one is given).
    """
    if stream is not None:
        return _on_stream(stream, lambda: layer_norm(x, weight, bias, eps=eps, out=out), x, weight, bias, out)
    device = torch.cuda.current_device()
    code, ldx, w_code, ldy = _forward(device, _meta(x), _meta(weight), _meta(bias), _meta(out))
    rows, d = x.shape
    if out is None:
        out = torch.empty((rows, d), dtype=x.dtype, device=device)
    mean = torch.empty(rows, dtype=_F32, device=device)
    rstd = torch.empty(rows, dtype=_F32, device=device)
    n = _pack(rows, d, x.data_ptr(), ldx, 0 if weight is None else weight.data_ptr(), 0 if bias is None else bias.data_ptr(),
              out.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0, eps, code, w_code, 0, 0)
    st = load_library().dgl_layer_norm(n, torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_layer_norm")
    return out, mean, rstd


@functools.lru_cache(maxsize=1024)
def _gradient(device, dy, x, mean, rstd, weight, need_dx, need_dw, need_db, dweight, dbias, dw_dtype, accumulate):
    code, ldx = _matrix(x, "x", device)
    rows, d = x[2]
    lddy = _matrix(dy, "dy", device, x[2], x[1])[1]
    _vector(mean, "mean", device, rows, _F32)
    _vector(rstd, "rstd", device, rows, _F32)
    w_code = _columns(device, d, weight, None)
    if not (need_dx or need_dw or need_db):
        raise ValueError("a call computes dx, dweight, dbias or some of them")
    if accumulate and not (need_dw or need_db):
        raise ValueError("accumulate adds to dweight and dbias, which are not asked for")
    if dw_dtype not in _TYPES:
        raise ValueError("dw_dtype must be OUT_BF16 or OUT_F32")
    given = [(m, name) for m, name in ((dweight, "dweight"), (dbias, "dbias")) if m is not None]
    for meta, name in given:
        _here(meta, name, device)
        dw_dtype = _type(meta, name)
    for meta, name, need in ((dweight, "dweight", need_dw), (dbias, "dbias", need_db)):
        if meta is None:
            if need and accumulate:
                raise ValueError(f"accumulate adds to the fp32 {name} that is passed in")
            continue
        if not need:
            raise ValueError(f"{name} is given but not asked for")
        if meta[1] != _TYPES[dw_dtype]:
            raise TypeError("dweight and dbias must have the same type")
        _vector(meta, name, device, d, meta[1])
    size = max(1, dgl_layer_norm_workspace(NormDesc(rows=rows, d=d))) if need_dw or need_db else 0
    return code, ldx, lddy, w_code, dw_dtype, size


def layer_norm_grad(dy, x, mean, rstd, weight=None, *, need_dx=True, need_dw=True, need_db=True, dweight=None,
                    dbias=None, dw_dtype=OUT_F32, accumulate=False, workspace=None, stream=None):
    """The gradient of layer_norm: (dx, dweight, dbias), None for those that are not needed.

    dy [rows, d] of x's type; mean and rstd as layer_norm returned them.  dx is
    of x's type; dweight and dbias [d] are fp32 or bf16 (dw_dtype, or the type of those passed
    in, which must be the same; accumulate adds to fp32 ones).  workspace: a
    CUDA buffer of at least dgl_layer_norm_workspace bytes, made when None.
    """
    if stream is not None:
        return _on_stream(stream, lambda: layer_norm_grad(
            dy, x, mean, rstd, weight, need_dx=need_dx, need_dw=need_dw, need_db=need_db, dweight=dweight, dbias=dbias,
            dw_dtype=dw_dtype, accumulate=accumulate, workspace=workspace),
            dy, x, mean, rstd, weight, dweight, dbias, workspace)
    device = torch.cuda.current_device()
    code, ldx, lddy, w_code, dw_dtype, size = _gradient(
        device, _meta(dy), _meta(x), _meta(mean), _meta(rstd), _meta(weight), need_dx, need_dw, need_db, _meta(dweight),
        _meta(dbias), dw_dtype, accumulate)
    rows, d = x.shape
    dx = torch.empty((rows, d), dtype=x.dtype, device=device) if need_dx else None
    if need_dw and dweight is None:
        dweight = torch.empty(d, dtype=_TYPES[dw_dtype], device=device)
    if need_db and dbias is None:
        dbias = torch.empty(d, dtype=_TYPES[dw_dtype], device=device)
    at = 0
    if size:
        if workspace is None:
            workspace = torch.empty(size, dtype=torch.uint8, device=device)
        else:
            _buffer(workspace, device)
            size = workspace.nbytes
        at = workspace.data_ptr()
    n = _pack(rows, d, x.data_ptr(), ldx, 0 if weight is None else weight.data_ptr(), 0, 0, 0, mean.data_ptr(),
              rstd.data_ptr(), dy.data_ptr(), lddy, dx.data_ptr() if need_dx else 0, d, dweight.data_ptr() if need_dw else 0,
              dbias.data_ptr() if need_db else 0, at, size, 0.0, code, w_code, dw_dtype, 1 if accumulate else 0)
    st = load_library().dgl_layer_norm_grad(n, torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_layer_norm_grad")
    return dx, dweight, dbias
