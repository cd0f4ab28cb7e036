"""The head losses on a stream that is not the one their tensors were made on: the
memory of a tensor that the caller drops after the call is not handed out again
before that stream is done with it."""
import gc

import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from tests.test_gpu_head import DEV, _inputs, _status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("op", ["xent", "distill"])
def test_dropped_tensors_are_kept_for_the_stream(op):
    T, V, d = 700, 3000, 256
    X, W, target, grad = _inputs(T, V, d)
    names = dict(X=X, W=W, target=target, grad=grad, dW=torch.zeros(V, d, device=DEV),
                 indices=target[:, None].contiguous(), logits=torch.zeros(T, 1, device=DEV),
                 teacher_lse=torch.zeros(T, device=DEV))

    def call(t, stream, workspace):
        if op == "xent":
            return dgl.linear_cross_entropy(t["X"], t["W"], t["target"], t["grad"], dW=t["dW"], stream=stream,
                                            workspace=workspace)
        return dgl.linear_distill(t["X"], t["W"], t["indices"], t["logits"], t["grad"], teacher_lse=t["teacher_lse"],
                                  dW=t["dW"], stream=stream, workspace=workspace)

    h = dgl.HeadDesc(T=T, V=V, d=d, grad=1, dX=1, dW=1, dw_dtype=dgl.OUT_F32)
    size = dgl.dgl_head_workspace(h, 0 if op == "xent" else 1)[1]
    want = [t.clone() for t in call(names, None, torch.empty(size, dtype=torch.uint8, device=DEV))]
    side = torch.cuda.Stream()
    mine = {n: t.clone() for n, t in names.items()}
    workspace = torch.empty(size, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    used = {"X", "W", "grad", "dW"} | ({"target"} if op == "xent" else {"indices", "logits", "teacher_lse"})
    kept = {mine[n].untyped_storage().data_ptr(): mine[n].nbytes for n in used}
    kept[workspace.untyped_storage().data_ptr()] = workspace.nbytes
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)  # some tenths of a second during which the call waits
    loss, lse, dX, _ = call(mine, side, workspace)
    assert not side.query(), "the stream was done too early to show anything"
    del mine, workspace, _
    gc.collect()
    # what the allocator hands out now on the current stream does not overlap what the call still uses
    fresh = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in list(kept.values()) * 2]
    for f in fresh:
        at = f.data_ptr()
        assert all(at + f.nbytes <= p or p + n <= at for p, n in kept.items()), "memory in use was handed out again"
        f.fill_(255)
    side.synchronize()
    _status()
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1]) and torch.equal(dX, want[2])
