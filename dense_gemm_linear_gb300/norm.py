"""Layer norm on torch CUDA tensors (dgl_layer_norm, dgl_layer_norm_grad).

The helpers check their arguments, allocate what is not passed in with torch,
and make one call of the library on torch's current stream.  The tensors are on
the current device, where the library launches.
"""
from __future__ import annotations

import functools

import torch

from . import OUT_BF16, OUT_F32, NormDesc, _check, dgl_layer_norm_workspace, load_library
from .head import _byref, _not_here, _on_stream, _packed, _rows

_F32 = torch.float32
_CODES = {torch.bfloat16: OUT_BF16, torch.float32: OUT_F32}


def _code(t, name):
    code = _CODES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if code is None:
        raise TypeError(f"{name} must be a bf16 or fp32 CUDA tensor")
    return code


def _matrix(t, name):
    """The type code and the extents of a matrix."""
    code = _code(t, name)
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    return code, *t.shape


def _vectors(d, device, **vectors):
    """Addresses of the weight and the bias (None where there is none), and their type."""
    at, code = [], OUT_F32
    first = None
    for name, t in vectors.items():
        if t is None:
            at.append(None)
            continue
        code = _code(t, name)
        if first is not None and first.dtype != t.dtype:
            raise TypeError("weight and bias must have the same type")
        first = t
        at.append(_packed(t, name, t.dtype, (d,), device))
    return at, code


@functools.lru_cache(maxsize=256)
def _workspace_bytes(rows, d):
    return dgl_layer_norm_workspace(NormDesc(rows=rows, d=d))


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, out=None, stream=None):
    """y = (x - mean) rstd weight + bias over the rows of x, with the statistics that the gradient reads.

    x [rows, d] bf16 or fp32 (rows may be strided); weight and bias [d], bf16 or
    fp32, or None.  Returns (y, mean, rstd): y of x's type (or `out`, which may be x),
    mean and rstd fp32 [rows].  All tensors are on the current device (stream's,
    when one is given).
    """
    if stream is not None:
        return _on_stream(stream, lambda: layer_norm(x, weight, bias, eps=eps, out=out), x, weight, bias, out)
    code, rows, d = _matrix(x, "x")
    device = torch.cuda.current_device()
    ldx = _rows(x, "x", x.dtype, (rows, d), device)
    (at_w, at_b), w_code = _vectors(d, device, weight=weight, bias=bias)
    if out is None:
        out = torch.empty((rows, d), dtype=x.dtype, device=device)
        ldy = d
    else:
        ldy = _rows(out, "out", x.dtype, (rows, d), device)
    mean = torch.empty(rows, dtype=_F32, device=device)
    rstd = torch.empty(rows, dtype=_F32, device=device)
    n = NormDesc(rows, d, x.data_ptr(), ldx, at_w, at_b, out.data_ptr(), ldy, mean.data_ptr(), rstd.data_ptr(),
                 eps=eps, x_dtype=code, w_dtype=w_code)
    st = load_library().dgl_layer_norm(_byref(n), torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_layer_norm")
    return out, mean, rstd


def _sums(given, name, d, want, dw_dtype, accumulate, device):
    """dweight or dbias: the tensor, made when it is None, or None when it is not wanted."""
    if not want:
        if given is not None:
            raise ValueError(f"{name} is given but not asked for")
        return None
    if given is None:
        if accumulate:
            raise ValueError(f"accumulate adds to the fp32 {name} that is passed in")
        return torch.empty(d, dtype=_F32 if dw_dtype == OUT_F32 else torch.bfloat16, device=device)
    _packed(given, name, given.dtype, (d,), device)
    return given


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
    code, rows, d = _matrix(x, "x")
    device = torch.cuda.current_device()
    ldx = _rows(x, "x", x.dtype, (rows, d), device)
    lddy = _rows(dy, "dy", x.dtype, (rows, d), device)
    at_mean = _packed(mean, "mean", _F32, (rows,), device)
    at_rstd = _packed(rstd, "rstd", _F32, (rows,), device)
    (at_w,), w_code = _vectors(d, device, weight=weight)
    if not (need_dx or need_dw or need_db):
        raise ValueError("a call computes dx, dweight, dbias or some of them")
    if dw_dtype not in (OUT_BF16, OUT_F32):
        raise ValueError("dw_dtype must be OUT_BF16 or OUT_F32")
    if accumulate and not (need_dw or need_db):
        raise ValueError("accumulate adds to dweight and dbias, which are not asked for")
    for name, t in (("dweight", dweight), ("dbias", dbias)):
        if t is not None:
            dw_dtype = _code(t, name)
    dweight = _sums(dweight, "dweight", d, need_dw, dw_dtype, accumulate, device)
    dbias = _sums(dbias, "dbias", d, need_db, dw_dtype, accumulate, device)
    if dweight is not None and dbias is not None and dweight.dtype != dbias.dtype:
        raise TypeError("dweight and dbias must have the same type")
    dx = torch.empty((rows, d), dtype=x.dtype, device=device) if need_dx else None
    size = 0
    if need_dw or need_db:
        if workspace is None:
            workspace = torch.empty(max(1, _workspace_bytes(rows, d)), dtype=torch.uint8, device=device)
        else:
            if not isinstance(workspace, torch.Tensor) or workspace.get_device() != device:
                _not_here(workspace, "workspace", device)
            if not workspace.is_contiguous():
                raise ValueError("workspace must be a contiguous CUDA tensor")
        size = workspace.nbytes
    n = NormDesc(rows, d, x.data_ptr(), ldx, at_w, None, None, 0, at_mean, at_rstd, dy.data_ptr(), lddy,
                 dx.data_ptr() if need_dx else None, d, dweight.data_ptr() if need_dw else None,
                 dbias.data_ptr() if need_db else None, workspace.data_ptr() if size else None, size, 0.0, code, w_code,
                 dw_dtype, 1 if accumulate else 0)
    st = load_library().dgl_layer_norm_grad(_byref(n), torch._C._cuda_getCurrentRawStream(device))
    if st:
        _check(st, "dgl_layer_norm_grad")
    return dx, dweight, dbias
