"""The head losses' host side: workspace sizes and refusals, which need no GPU
(every check comes before the first device call)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    from dense_gemm_linear_gb300 import _build
    _build.build()
    d.load_library()
    return d


def _head(dgl, **kw):
    h = dgl.HeadDesc()
    vals = dict(T=100, V=1000, d=64, X=0x10000, W=0x20000, loss=0x30000, lse=0x40000, grad=0x50000, dX=0x60000,
                dW=0x70000, ws=0x100000, ws_bytes=1 << 40, logit_scale=1.0, dw_dtype=dgl.OUT_F32)
    vals.update(kw)
    for k, v in vals.items():
        setattr(h, k, v)
    return h


REFUSED = [
    (dict(T=-1), "ARG"), (dict(V=0), "ARG"), (dict(d=0), "ARG"), (dict(d=-8), "ARG"), (dict(d=60), "ALIGN"),
    (dict(T=1 << 31), "SHAPE"), (dict(V=1 << 31), "SHAPE"), (dict(X=0), "ARG"), (dict(W=0), "ARG"),
    (dict(loss=0), "ARG"), (dict(grad=0), "ARG"), (dict(dX=0, dW=0), "ARG"), (dict(X=0x10008), "ALIGN"),
    (dict(W=0x20002), "ALIGN"), (dict(dX=0x60004), "ALIGN"), (dict(dW=0x70008), "ALIGN"), (dict(ldx=60), "ARG"),
    (dict(ldx=68), "ALIGN"), (dict(ldw=8), "ARG"), (dict(lddx=66), "ALIGN"), (dict(lddw=32), "ARG"),
    (dict(ldx=1 << 31), "SHAPE"), (dict(loss=0x30002), "ALIGN"), (dict(grad=0x50001), "ALIGN"), (dict(ws=0), "ARG"),
    (dict(ws=0x100010), "ALIGN"), (dict(ws_bytes=1000), "ARG"), (dict(logit_scale=float("nan")), "ARG"),
    (dict(logit_scale=float("inf")), "ARG"), (dict(dw_dtype=2), "ARG"), (dict(accumulate=2), "ARG"),
    (dict(accumulate=1, dw_dtype=0), "ARG"), (dict(accumulate=1, dW=0), "ARG"),
]


@pytest.mark.parametrize("change,code", REFUSED)
def test_refusals(dgl, change, code):
    want = getattr(dgl, "DGL_ERR_" + code)
    h = _head(dgl, **change)
    assert dgl.dgl_linear_xent(h, 0x80000) == want
    assert dgl.dgl_linear_distill(h, 0x80000, 0x90000, None, 4) == want


def test_refusals_of_targets(dgl):
    h = _head(dgl)
    assert dgl.dgl_linear_xent(h, None) == dgl.DGL_ERR_ARG
    assert dgl.dgl_linear_xent(h, 0x80004) == dgl.DGL_ERR_ALIGN
    assert dgl.dgl_linear_distill(h, None, 0x90000, None, 4) == dgl.DGL_ERR_ARG
    assert dgl.dgl_linear_distill(h, 0x80000, None, None, 4) == dgl.DGL_ERR_ARG
    assert dgl.dgl_linear_distill(h, 0x80000, 0x90002, None, 4) == dgl.DGL_ERR_ALIGN
    assert dgl.dgl_linear_distill(h, 0x80000, 0x90000, 0x90002, 4) == dgl.DGL_ERR_ALIGN
    for k in (0, -1, dgl.DISTILL_MAX_K + 1):
        assert dgl.dgl_linear_distill(h, 0x80000, 0x90000, None, k) == dgl.DGL_ERR_ARG
    for temp in (0.0, -1.0, float("nan"), float("inf")):
        assert dgl.dgl_linear_distill(h, 0x80000, 0x90000, None, 4, temp) == dgl.DGL_ERR_ARG
    assert dgl.load_library().dgl_linear_xent(None, 0x80000, -100, None) == dgl.DGL_ERR_ARG
    assert dgl.load_library().dgl_linear_distill(None, 0x80000, 0x90000, None, 4, 1.0, None) == dgl.DGL_ERR_ARG


def test_workspace_sizes(dgl):
    """The minimum does not grow with T once the call takes chunks; the best
    stays within a few GiB however many tokens there are; forward needs less."""
    for V, d, dw in ((50257, 512, 0), (32000, 4096, 1), (7, 8, 0), (262144, 2048, 0)):
        sizes = [dgl.dgl_head_workspace(_head(dgl, T=T, V=V, d=d, dw_dtype=dw)) for T in (1, 128, 4096, 1 << 20, 1 << 24)]
        assert all(0 < low for low, _ in sizes)
        assert sizes[3][0] == sizes[4][0]
        sums = 4 * V * d + (1 << 20)
        assert all(best <= (4 << 30) + sums for _, best in sizes)
        assert all(a[1] <= b[1] + sums for a, b in zip(sizes, sizes[1:]))
        fwd = dgl.dgl_head_workspace(_head(dgl, T=4096, V=V, d=d, grad=0, dX=0, dW=0))
        assert fwd[1] <= sizes[2][1]
    with pytest.raises(dgl.DglError):
        dgl.dgl_head_workspace(_head(dgl, V=0))
    low, best = ctypes.c_int64(), ctypes.c_int64()
    lib = dgl.load_library()
    assert lib.dgl_head_workspace(None, 0, ctypes.byref(low), ctypes.byref(best)) == dgl.DGL_ERR_ARG
    assert lib.dgl_head_workspace(ctypes.byref(_head(dgl)), 0, None, ctypes.byref(best)) == dgl.DGL_ERR_ARG
    assert lib.dgl_head_workspace(ctypes.byref(_head(dgl)), 129, ctypes.byref(low), ctypes.byref(best)) == dgl.DGL_ERR_ARG


def test_no_tokens_needs_no_buffers(dgl):
    """T == 0 passes the checks without X, loss, targets or a workspace (and
    then fails only for want of a device, where there is none)."""
    h = _head(dgl, T=0, X=0, loss=0, lse=0, ws=0, ws_bytes=0, accumulate=1)
    import torch
    want = dgl.DGL_OK if torch.cuda.is_available() else dgl.DGL_ERR_CUDA
    assert dgl.dgl_linear_xent(h, None) in (want, dgl.DGL_ERR_UNSUPPORTED)
