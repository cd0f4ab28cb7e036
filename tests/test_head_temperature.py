"""A temperature whose reciprocal is past fp32's range is refused before anything is
launched: the teacher's logits are multiplied by it."""
import pytest

import dense_gemm_linear_gb300 as dgl
from tests.test_head_host import _head


@pytest.fixture(scope="module", autouse=True)
def built():
    from dense_gemm_linear_gb300 import _build
    _build.build()
    dgl.load_library()


@pytest.mark.parametrize("temperature,scale", [(1e-39, 1e-30), (1e-45, 0.0), (2.9e-39, -1e-20)])
def test_reciprocal_not_finite(temperature, scale):
    h = _head(dgl, logit_scale=scale)
    assert dgl.dgl_linear_distill(h, 0x80000, 0x90000, None, 4, temperature) == dgl.DGL_ERR_ARG
