"""dgl_head_workspace counts what the asked-for gradients need: the copy of X's rows
only with dW, the scratch of dX's ranges only with dX (pure host logic)."""
import pytest


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    from dense_gemm_linear_gb300 import _build
    _build.build()
    d.load_library()
    return d


SPLIT_BYTES = 160 * 128 * 256 * 4  # a partial tile for each CTA


def _sizes(dgl, T, V, d, dx, dw, k, dw_dtype):
    h = dgl.HeadDesc(T=T, V=V, d=d, grad=1, dX=dx, dW=dw, dw_dtype=dw_dtype)
    return dgl.dgl_head_workspace(h, k)


@pytest.mark.parametrize("k", [0, 9])
@pytest.mark.parametrize("T,V,d", [(1, 7, 8), (1000, 50257, 512), (4096, 32000, 4096), (20000, 50257, 64)])
def test_scratch_of_one_gradient(dgl, T, V, d, k):
    # (an fp32 dW needs no sums of its own, so that the two copies are what is left)
    both, dx, dw = (_sizes(dgl, T, V, d, a, b, k, dgl.OUT_F32) for a, b in ((1, 1), (1, 0), (0, 1)))
    rows_least = 128
    rows_most = min(-(-T // 128) * 128, max(128, (1 << 30) // (-(-V // 64) * 64 * 2) // 128 * 128))
    for i, rows in ((0, min(rows_least, rows_most)), (1, rows_most)):
        assert both[i] - dx[i] == -(-rows * d * 2 // 256) * 256
        assert both[i] - dw[i] >= SPLIT_BYTES


def test_scratch_of_none_for_a_forward_pass(dgl):
    fwd = dgl.dgl_head_workspace(dgl.HeadDesc(T=1000, V=50257, d=512), 0)
    for dx, dw in ((1, 0), (0, 1)):
        assert fwd[1] < _sizes(dgl, 1000, 50257, 512, dx, dw, 0, dgl.OUT_F32)[1]
