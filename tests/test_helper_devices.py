"""The torch helpers of the GEMMs launch on the current device: tensors and streams
of any other, and an `out` in host memory, are refused before the library is
called.  The tensors are stand-ins in host memory that say which device they
are on."""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl

M, N, K = 8, 24, 128
SHAPES = {
    "gemm_bf16": dict(A=((M, K), torch.bfloat16), B=((N, K), torch.bfloat16)),
    "gemm_fp8": dict(A=((M, K), torch.float8_e4m3fn), B=((N, K), torch.float8_e4m3fn), sa=((M,), torch.float32),
                     sb=((N,), torch.float32)),
    "gemm_mxfp4": dict(A=((M, K // 2), torch.uint8), B=((N, K // 2), torch.uint8), sfa=((M, K // 32), torch.uint8),
                       sfb=((N, K // 32), torch.uint8)),
    "gemm_w4a8": dict(A=((M, K), torch.float8_e4m3fn), B=((N, K // 2), torch.uint8), sa=((M,), torch.float32),
                      sb=((N,), torch.float32)),
    "linear": dict(A=((M, K), torch.bfloat16), B=((N, K), torch.bfloat16), bias=((N,), torch.float32)),
}


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: self.index >= 0)
    device = property(lambda self: torch.device("cuda", self.index) if self.index >= 0 else torch.device("cpu"))

    def get_device(self):
        return self.index


class Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 0


class Called(Exception):
    pass


@pytest.fixture()
def current(monkeypatch):
    class Library:
        def __getattr__(self, name):
            raise Called(name)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(0))
    monkeypatch.setattr(dgl, "load_library", lambda path=None: Library())


def _call(name, where, stream=None):
    args = {}
    for key, (shape, dtype) in dict(SHAPES[name], out=((M, N), torch.bfloat16)).items():
        args[key] = torch.empty(shape, dtype=dtype).as_subclass(OnDevice)
        args[key].index = where.get(key, 0)
    if name in ("gemm_mxfp4", "gemm_w4a8"):
        args["K"] = K
    return getattr(dgl, name)(**args, stream=stream)


@pytest.mark.parametrize("name", SHAPES)
def test_one_tensor_on_another_device(current, name):
    with pytest.raises(Called):
        _call(name, {})
    with pytest.raises(Called):
        _call(name, {}, Stream(0))
    for key in list(SHAPES[name]) + ["out"]:
        with pytest.raises(ValueError, match="cuda:1"):
            _call(name, {key: 1})
    with pytest.raises(ValueError, match="cpu"):
        _call(name, {"out": -1})


@pytest.mark.parametrize("name", SHAPES)
def test_a_device_that_is_not_current(current, name):
    with pytest.raises(ValueError, match="cuda:1"):
        _call(name, dict.fromkeys(list(SHAPES[name]) + ["out"], 1))
    with pytest.raises(ValueError, match="cuda:1"):
        _call(name, {}, Stream(1))
