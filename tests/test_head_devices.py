"""The head losses' helpers launch on the current device: tensors of any other are
refused before the library is called.  The tensors are stand-ins that lie in
host memory and say which device they are on."""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from dense_gemm_linear_gb300 import head

BF16, F32, I64 = torch.bfloat16, torch.float32, torch.int64
T, V, D, K = 6, 40, 16, 3


class OnDevice(torch.Tensor):
    is_cuda = property(lambda self: self.index >= 0)

    def get_device(self):
        return self.index


def _on(index, *shape, dtype):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    t.index = index
    return t


class Called(Exception):
    pass


@pytest.fixture()
def current(monkeypatch):
    """Makes cuda:0 the current device; allocations go to host memory and a call of the library raises Called."""
    empty = torch.empty

    class Library:
        def __getattr__(self, name):
            raise Called(name)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(head, "load_library", lambda: Library())


def _arguments(where):
    """All tensors of a call, on cuda:0 but for those named in `where`."""
    shapes = dict(X=((T, D), BF16), W=((V, D), BF16), grad=((T,), F32), dW=((V, D), F32), target=((T,), I64),
                  indices=((T, K), I64), logits=((T, K), F32), teacher_lse=((T,), F32), workspace=((1 << 26,), torch.uint8))
    return {name: _on(where.get(name, 0), *shape, dtype=dtype) for name, (shape, dtype) in shapes.items()}


def _xent(where):
    a = _arguments(where)
    return dgl.linear_cross_entropy(a["X"], a["W"], a["target"], a["grad"], dW=a["dW"], workspace=a["workspace"])


def _distill(where):
    a = _arguments(where)
    return dgl.linear_distill(a["X"], a["W"], a["indices"], a["logits"], a["grad"], teacher_lse=a["teacher_lse"],
                              dW=a["dW"], workspace=a["workspace"])


CALLS = [(_xent, ["X", "W", "target", "grad", "dW", "workspace"]),
         (_distill, ["X", "W", "indices", "logits", "teacher_lse", "grad", "dW", "workspace"])]


@pytest.mark.parametrize("call,names", CALLS, ids=["xent", "distill"])
def test_one_tensor_on_another_device(current, call, names):
    with pytest.raises(Called):  # all on the current device: the library is reached
        call({})
    for name in names:
        with pytest.raises(ValueError, match="cuda:1"):
            call({name: 1})


@pytest.mark.parametrize("call,names", CALLS, ids=["xent", "distill"])
def test_all_tensors_on_a_device_that_is_not_current(current, call, names):
    with pytest.raises(ValueError, match="cuda:1"):
        call(dict.fromkeys(names, 1))


@pytest.mark.parametrize("call,names", CALLS, ids=["xent", "distill"])
def test_host_tensors(current, call, names):
    for name in names:
        with pytest.raises((TypeError, ValueError)):
            call({name: -1})
