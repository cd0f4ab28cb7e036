"""MN-major B (dgl_gemm_bf16_ex) on shapes whose plan is the 224-wide tile.

An MN-major B is loaded in boxes of 64 columns, and a CTA of a 224-wide pair
tile holds 112: such calls run on 256-wide tiles, and a forced 224-wide plan is
refused.  Tolerance as in the other layout tests."""
import pytest

import dense_gemm_linear_gb300 as dgl
from synthetic import make_case
from tests import gpu_util as gu
from tests.test_gpu_layouts import K_, MN_, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [(K_, MN_), (MN_, MN_)], ids=["dX", "dW"])
@pytest.mark.parametrize("m,n,K", [(3156, 392, 864), (2048, 4096, 256)])
def test_shapes_planned_224_wide(layout, m, n, K):
    assert dgl.plan(dgl.DTYPE_BF16, m, n, K, num_sms=152)["tile_n"] == 224
    case = make_case("bf16", m, n, K, out="bf16")
    Cbuf = _run(case, *layout)
    gu.assert_close_sampled(case, Cbuf, seed=3)


def test_forced_224_wide_plan_is_refused():
    plan = dgl.PlanInfo(path=dgl.PATH_TC, tile_m=256, tile_n=224)
    for a_major in (K_, MN_):
        # refused before any operand is read
        st = dgl.dgl_gemm_bf16_ex(a_major, MN_, 0x10000, 64, 0x20000, 448, 0x30000, 448, 64, 448, 64, dgl.OUT_BF16,
                                  plan, 0)
        assert st == dgl.DGL_ERR_UNSUPPORTED
