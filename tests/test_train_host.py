"""The host side of the embedding, the layer norm and AdamW: workspace sizes
and refusals, which need no GPU (every check comes before the first device
call), and the helpers' checks of their tensors."""
import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from dense_gemm_linear_gb300 import embed, norm, optim

# the addresses below are made up: none may ever reach a device
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for a machine without a GPU")
BF16, F32, I64, U8 = torch.bfloat16, torch.float32, torch.int64, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def library():
    from dense_gemm_linear_gb300 import _build
    _build.build()
    dgl.load_library()


def _norm(**kw):
    vals = dict(rows=100, d=64, x=0x10000, weight=0x20000, bias=0x30000, y=0x40000, mean=0x50000, rstd=0x60000,
                dy=0x70000, dx=0x80000, dweight=0x90000, dbias=0xa0000, ws=0x100000, ws_bytes=1 << 40, eps=1e-5,
                x_dtype=dgl.OUT_BF16, w_dtype=dgl.OUT_F32, dw_dtype=dgl.OUT_F32)
    vals.update(kw)
    return dgl.NormDesc(**vals)


def _embed(**kw):
    vals = dict(T=100, V=1000, d=64, tokens=0x10000, ignore_index=-100, W=0x20000, dW=0x30000, Y=0x40000, dY=0x50000,
                ws=0x100000, ws_bytes=1 << 40, scale=1.0, w_dtype=dgl.OUT_F32, y_dtype=dgl.OUT_BF16)
    vals.update(kw)
    return dgl.EmbedDesc(**vals)


# a change, the code, and the calls that it concerns (forward, gradient)
NORM = [
    (dict(rows=-1), "ARG", "fg"), (dict(d=0), "ARG", "fg"), (dict(d=-3), "ARG", "fg"), (dict(rows=1 << 31), "SHAPE", "fg"),
    (dict(rows=(1 << 31) - 1), "SHAPE", "fg"), (dict(d=1 << 28), "SHAPE", "fg"), (dict(x=0), "ARG", "fg"),
    (dict(y=0), "ARG", "f"), (dict(dy=0), "ARG", "g"), (dict(mean=0), "ARG", "g"), (dict(rstd=0), "ARG", "g"),
    (dict(dx=0, dweight=0, dbias=0), "ARG", "g"), (dict(x=0x10001), "ALIGN", "fg"), (dict(y=0x40001), "ALIGN", "f"),
    (dict(dy=0x70001), "ALIGN", "g"), (dict(dx=0x80001), "ALIGN", "g"), (dict(weight=0x20002), "ALIGN", "fg"),
    (dict(bias=0x30002), "ALIGN", "fg"), (dict(mean=0x50002), "ALIGN", "fg"), (dict(rstd=0x60001), "ALIGN", "fg"),
    (dict(dweight=0x90002), "ALIGN", "g"), (dict(dbias=0xa0002), "ALIGN", "g"), (dict(ldx=63), "ARG", "fg"),
    (dict(ldy=1), "ARG", "f"), (dict(lddy=-64), "ARG", "g"), (dict(lddx=10), "ARG", "g"),
    (dict(ldx=1 << 31), "SHAPE", "fg"), (dict(ws=0), "ARG", "g"), (dict(ws=0x100010), "ALIGN", "g"),
    (dict(ws_bytes=100), "ARG", "g"), (dict(eps=-1.0), "ARG", "f"), (dict(eps=float("nan")), "ARG", "f"),
    (dict(eps=float("inf")), "ARG", "f"), (dict(x_dtype=2), "ARG", "fg"), (dict(w_dtype=-1), "ARG", "fg"),
    (dict(dw_dtype=5), "ARG", "fg"), (dict(accumulate=2), "ARG", "g"), (dict(accumulate=1, dw_dtype=0), "ARG", "g"),
    (dict(accumulate=1, dweight=0, dbias=0), "ARG", "g"),
]


@pytest.mark.parametrize("change,code,calls", NORM)
def test_norm_refusals(change, code, calls):
    want = getattr(dgl, "DGL_ERR_" + code)
    if "f" in calls:
        assert dgl.dgl_layer_norm(_norm(**change)) == want
    if "g" in calls:
        assert dgl.dgl_layer_norm_grad(_norm(**change)) == want


EMBED = [
    (dict(T=-1), "ARG", "fg"), (dict(V=0), "ARG", "fg"), (dict(d=0), "ARG", "fg"), (dict(T=1 << 31), "SHAPE", "fg"),
    (dict(V=(1 << 31) - 5), "SHAPE", "fg"), (dict(d=1 << 28), "SHAPE", "fg"), (dict(tokens=0), "ARG", "fg"),
    (dict(W=0), "ARG", "f"), (dict(Y=0), "ARG", "f"), (dict(dW=0), "ARG", "g"), (dict(dY=0), "ARG", "g"),
    (dict(tokens=0x10004), "ALIGN", "fg"), (dict(W=0x20002), "ALIGN", "f"), (dict(Y=0x40001), "ALIGN", "f"),
    (dict(dW=0x30001), "ALIGN", "g"), (dict(dY=0x50001), "ALIGN", "g"), (dict(ldw=32), "ARG", "fg"),
    (dict(ldy=-1), "ARG", "fg"), (dict(ldw=1 << 31), "SHAPE", "fg"), (dict(ws=0), "ARG", "g"),
    (dict(ws=0x100080), "ALIGN", "g"), (dict(ws_bytes=64), "ARG", "g"), (dict(scale=float("nan")), "ARG", "fg"),
    (dict(scale=float("inf")), "ARG", "fg"), (dict(w_dtype=3), "ARG", "fg"), (dict(y_dtype=-1), "ARG", "fg"),
    (dict(accumulate=2), "ARG", "g"), (dict(accumulate=1, w_dtype=0), "ARG", "g"),
]


@pytest.mark.parametrize("change,code,calls", EMBED)
def test_embedding_refusals(change, code, calls):
    want = getattr(dgl, "DGL_ERR_" + code)
    if "f" in calls:
        assert dgl.dgl_embedding(_embed(**change)) == want
    if "g" in calls:
        assert dgl.dgl_embedding_grad(_embed(**change)) == want


def _adam(tensor=(), **kw):
    vals = dict(steps=0x1000, ticket=0x2000, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, state_bits=8)
    vals.update(kw)
    t = dict(param=0x10000, grad=0x20000, exp_avg=0x40000, exp_avg_sq=0x50000, exp_avg_scale=0x60000,
             exp_avg_sq_scale=0x70000, n=1000, weight_decay=0.1, param_dtype=dgl.OUT_BF16, grad_dtype=dgl.OUT_F32)
    t.update(tensor)
    tensors = (dgl.AdamWTensor * 2)(dgl.AdamWTensor(**{**t, "param": 0x80000} if "param" not in dict(tensor) else t),
                                    dgl.AdamWTensor(**t))
    return dgl.dgl_adamw(dgl.AdamWDesc(**vals), tensors)


@pytest.mark.parametrize("change,code", [
    (dict(steps=0), "ARG"), (dict(ticket=0), "ARG"), (dict(steps=0x1004), "ALIGN"), (dict(ticket=0x2002), "ALIGN"),
    (dict(grad_scale=0x3001), "ALIGN"), (dict(lr_at=0x3002), "ALIGN"), (dict(lr=float("nan")), "ARG"),
    (dict(lr=float("inf")), "ARG"), (dict(beta1=1.0), "ARG"), (dict(beta1=-0.1), "ARG"), (dict(beta2=float("nan")), "ARG"),
    (dict(beta2=1.5), "ARG"), (dict(eps=-1e-8), "ARG"), (dict(eps=float("inf")), "ARG"), (dict(state_bits=4), "ARG"),
    (dict(state_bits=0), "ARG"),
])
def test_adamw_refusals(change, code):
    assert _adam(**change) == getattr(dgl, "DGL_ERR_" + code)


@pytest.mark.parametrize("change,code", [
    (dict(n=-1), "ARG"), (dict(n=(1 << 40) + 1), "SHAPE"), (dict(param=0), "ARG"), (dict(grad=0), "ARG"),
    (dict(exp_avg=0), "ARG"), (dict(exp_avg_sq=0), "ARG"), (dict(exp_avg_scale=0), "ARG"), (dict(exp_avg_sq_scale=0), "ARG"),
    (dict(master=0x30000, param_dtype=1), "ARG"), (dict(master=0x30002), "ALIGN"), (dict(param=0x10001), "ALIGN"),
    (dict(grad=0x20002), "ALIGN"), (dict(exp_avg_scale=0x60002), "ALIGN"), (dict(weight_decay=-0.1), "ARG"),
    (dict(weight_decay=float("nan")), "ARG"), (dict(param_dtype=2), "ARG"), (dict(grad_dtype=-1), "ARG"),
])
def test_adamw_tensor_refusals(change, code):
    assert _adam(tensor=change) == getattr(dgl, "DGL_ERR_" + code)
    assert _adam(tensor=dict(exp_avg=0x40002), state_bits=32) == dgl.DGL_ERR_ALIGN


def test_null_descriptors():
    lib = dgl.load_library()
    assert lib.dgl_layer_norm(None, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_layer_norm_grad(None, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_layer_norm_workspace(None, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_embedding(None, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_embedding_grad(None, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_embedding_workspace(None, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_adamw(None, None, 0, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_adamw(dgl.AdamWDesc(steps=8, ticket=4, state_bits=32), None, 3, None) == dgl.DGL_ERR_ARG
    assert lib.dgl_adamw(dgl.AdamWDesc(steps=8, ticket=4, state_bits=32), None, -1, None) == dgl.DGL_ERR_ARG


def test_workspace_sizes():
    """They grow with the problem no faster than it, and not at all past a grid's blocks or a sort's tokens."""
    for d in (8, 4096, 8192, 16384, 40000):
        sizes = [dgl.dgl_layer_norm_workspace(_norm(rows=r, d=d)) for r in (0, 1, 100, 10**5, 10**9)]
        assert sizes[0] == 0 and sizes[1] >= 8 * d and sizes[3] == sizes[4] and sizes == sorted(sizes)
        assert sizes[4] <= 160 * 8 * d
    for V, d, y in ((50257, 2048, 0), (32000, 4096, 1), (7, 8, 0), (262144, 64, 0)):
        sizes = [dgl.dgl_embedding_workspace(_embed(T=T, V=V, d=d, y_dtype=y)) for T in (0, 1, 1000, 131072, 10**8)]
        assert sizes[0] == 0 and sizes == sorted(sizes) and sizes[3] == sizes[4]
        sums = dgl.dgl_embedding_workspace(_embed(T=10**8, V=V, d=d, y_dtype=y, w_dtype=0))
        assert sums >= 4 * V * d and sums <= sizes[4] + 4 * V * d + 256
    with pytest.raises(dgl.DglError):
        dgl.dgl_layer_norm_workspace(_norm(d=0))
    with pytest.raises(dgl.DglError):
        dgl.dgl_embedding_workspace(_embed(V=0))


# ---- the helpers, on stand-ins that lie in host memory and say which device they are on

class OnDevice(torch.Tensor):
    index = 0  # of those that are made from others
    is_cuda = property(lambda self: self.index >= 0)

    def get_device(self):
        return self.index


def _on(index, *shape, dtype=F32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(OnDevice)
    t.index = index
    return t


class Called(Exception):
    pass


@pytest.fixture()
def current(monkeypatch):
    """Makes cuda:0 the current device; allocations go to host memory and a call of the library raises Called."""
    empty, zeros = torch.empty, torch.zeros

    def here(t):
        t = t.as_subclass(OnDevice)
        t.index = 0
        return t

    class Library:
        def __getattr__(self, name):
            raise Called(name)

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: here(empty(*a, **k)))
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: here(zeros(*a, **k)))
    for module in (norm, embed, optim):
        monkeypatch.setattr(module, "load_library", lambda: Library())


T, V, D = 6, 40, 16


def _arguments(where=None):
    shapes = dict(x=((T, D), BF16), dy=((T, D), BF16), weight=((D,), F32), bias=((D,), F32), mean=((T,), F32),
                  rstd=((T,), F32), dweight=((D,), F32), dbias=((D,), F32), out=((T, D), BF16), tokens=((T,), I64),
                  W=((V, D), BF16), dY=((T, D), BF16), dW=((V, D), F32), p=((5, 3), BF16), g=((5, 3), F32),
                  master=((5, 3), F32), m=((15,), F32), v=((15,), F32), steps=((1,), I64), lr=((1,), F32),
                  grad_scale=((1,), F32), workspace=((1 << 22,), U8))
    made = {k: _on((where or {}).get(k, 0), *shape, dtype=dtype) for k, (shape, dtype) in shapes.items()}
    return made


def _call_norm(a):
    dgl.layer_norm(a["x"], a["weight"], a["bias"], out=a["out"])


def _call_norm_grad(a):
    dgl.layer_norm_grad(a["dy"], a["x"], a["mean"], a["rstd"], a["weight"], dweight=a["dweight"], dbias=a["dbias"],
                        accumulate=True, workspace=a["workspace"])


def _call_embedding(a):
    dgl.embedding(a["tokens"], a["W"], out=a["out"])


def _call_embedding_grad(a):
    dgl.embedding_grad(a["tokens"], a["dY"], V, dW=a["dW"], accumulate=True, workspace=a["workspace"])


def _call_adamw(a):
    opt = dgl.AdamW([a["p"]], [a["g"]], master=[a["master"]], exp_avg=[a["m"]], exp_avg_sq=[a["v"]], steps=a["steps"])
    opt.step(lr=a["lr"], grad_scale=a["grad_scale"])


CALLS = [(_call_norm, ["x", "weight", "bias", "out"]),
         (_call_norm_grad, ["dy", "x", "mean", "rstd", "weight", "dweight", "dbias", "workspace"]),
         (_call_embedding, ["tokens", "W", "out"]), (_call_embedding_grad, ["tokens", "dY", "dW", "workspace"]),
         (_call_adamw, ["p", "g", "master", "m", "v", "steps", "lr", "grad_scale"])]
IDS = ["norm", "norm_grad", "embedding", "embedding_grad", "adamw"]


@pytest.fixture()
def raw_stream(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)


@pytest.mark.parametrize("call,names", CALLS, ids=IDS)
def test_tensors_of_another_device(current, raw_stream, call, names):
    with pytest.raises(Called):  # all on the current device: the library is reached
        call(_arguments())
    for name in names:
        with pytest.raises(ValueError, match="cuda:1"):
            call(_arguments({name: 1}))
        with pytest.raises((TypeError, ValueError)):  # host tensors
            call(_arguments({name: -1}))


@pytest.mark.parametrize("call,names", CALLS, ids=IDS)
def test_tensors_of_another_shape_or_type(current, raw_stream, call, names):
    for name in names:
        if name == "workspace":
            continue
        a = _arguments()
        shape = list(a[name].shape)
        shape[-1] += 1
        a[name] = _on(0, *shape, dtype=a[name].dtype)
        # (one tensor alone may have any width; the others then differ from it)
        with pytest.raises((TypeError, ValueError)):
            call(a)
        a = _arguments()
        a[name] = _on(0, *a[name].shape, dtype=torch.float16)
        with pytest.raises(TypeError):
            call(a)


def test_helper_refusals(current, raw_stream):
    a = _arguments()
    x, w, dy, mean, rstd = a["x"], a["weight"], a["dy"], a["mean"], a["rstd"]
    for bad in (lambda: dgl.layer_norm(x[0]), lambda: dgl.layer_norm(x.t()), lambda: dgl.layer_norm(x[:1].expand(T, D)),
                lambda: dgl.layer_norm(x, w, a["bias"].bfloat16()), lambda: dgl.layer_norm(x, w[::2]),
                lambda: dgl.layer_norm_grad(dy, x, mean, rstd, w, need_dx=False, need_dw=False, need_db=False),
                lambda: dgl.layer_norm_grad(dy, x, mean, rstd, w, dw_dtype=7),
                lambda: dgl.layer_norm_grad(dy, x, mean, rstd, w, accumulate=True),
                lambda: dgl.layer_norm_grad(dy, x, mean, rstd, w, need_dw=False, dweight=a["dweight"]),
                lambda: dgl.layer_norm_grad(dy, x, mean, rstd, w, dweight=a["dweight"], dbias=_on(0, D, dtype=BF16)),
                lambda: dgl.layer_norm_grad(dy, x, mean, rstd, w, need_dw=False, need_db=False, accumulate=True),
                lambda: dgl.embedding(a["tokens"][:, None], a["W"]), lambda: dgl.embedding(a["tokens"], a["W"], out_dtype=3),
                lambda: dgl.embedding(a["tokens"], a["W"], out=a["out"], out_dtype=dgl.OUT_F32),
                lambda: dgl.embedding(a["tokens"], a["W"], ignore_index=None),
                lambda: dgl.embedding(a["tokens"], a["W"], ignore_index=1 << 63),
                lambda: dgl.layer_norm(x, w, eps="1e-5"),
                lambda: dgl.embedding_grad(a["tokens"], a["dY"], V, accumulate=True),
                lambda: dgl.embedding_grad(a["tokens"], a["dY"], V, dw_dtype=9),
                lambda: dgl.embedding_grad(a["tokens"], a["dY"], V + 1, dW=a["dW"]),
                lambda: dgl.AdamW([a["p"]], [a["g"]], state_bits=4), lambda: dgl.AdamW([a["p"]], []),
                lambda: dgl.AdamW([a["p"]], [a["g"]], weight_decay=[0.1, 0.1]),
                lambda: dgl.AdamW([a["p"]], [a["g"]], exp_avg=[]),
                lambda: dgl.AdamW([a["p"]], [a["g"]], exp_avg_scale=[a["m"]]),
                lambda: dgl.AdamW([a["g"]], [a["g"]], master=[a["master"]]),
                lambda: dgl.AdamW([a["p"], a["p"]], [a["g"], a["g"]]),
                lambda: dgl.AdamW([a["p"], a["p"].clone()], [a["g"], a["g"]], master=[a["master"]] * 2),
                lambda: dgl.AdamW([a["p"]], [a["g"]], exp_avg=[a["m"]], exp_avg_sq=[a["m"]], steps=a["steps"]),
                lambda: dgl.AdamW([a["p"].t()], [a["g"].t()]), lambda: dgl.AdamW([a["p"]]).step()):
        with pytest.raises((TypeError, ValueError)):
            bad()
