"""Which memory a step of AdamW reaches when its tensors have been replaced, and tensors that overlap: on stand-ins in
host memory, with a library that notes what it is given."""
import ctypes

import pytest
import torch

import dense_gemm_linear_gb300 as dgl
from dense_gemm_linear_gb300 import optim

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="for a machine without a GPU")
BF16, F32, I64, E4M3, E5M2 = torch.bfloat16, torch.float32, torch.int64, torch.float8_e4m3fn, torch.float8_e5m2
SIZES = (200, 15)


class OnDevice(torch.Tensor):
    index = 0
    is_cuda = property(lambda self: self.index >= 0)

    def get_device(self):
        return self.index


def here(t):
    return t.as_subclass(OnDevice)


def some(n, dtype=F32):
    return here(torch.ones(n).to(dtype))


@pytest.fixture()
def calls(monkeypatch):
    """The tables and step counters that reach dgl_adamw, one entry a call."""
    made = []

    class Library:
        def dgl_adamw(self, desc, table, count, stream):
            desc = ctypes.cast(desc, ctypes.POINTER(dgl.AdamWDesc)).contents
            names = [name for name, _ in dgl.AdamWTensor._fields_]
            made.append(([{name: getattr(table[i], name) for name in names} for i in range(count)], desc.steps))
            return dgl.DGL_OK

    zeros = torch.zeros
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: here(zeros(*a, **k)))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    monkeypatch.setattr(optim, "load_library", lambda: Library())
    return made


def make(bits=8, **given):
    params = [some(n, BF16) for n in SIZES]
    grads = [some(n) for n in SIZES]
    return dgl.AdamW(params, grads, master=True, state_bits=bits, **given), params, grads


def expect(call, opt):
    """A call is given the memory of what the optimizer has now."""
    table, steps = call
    assert steps == opt.steps.data_ptr()
    for i, row in enumerate(table):
        assert row["param"] == opt.params[i].data_ptr() and row["grad"] == opt.grads[i].data_ptr()
        assert row["master"] == opt.master[i].data_ptr()
        for name in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
            held = getattr(opt, name)
            assert row[name] == (None if held is None else held[i].data_ptr())


@pytest.mark.parametrize("bits", [8, 32])
def test_params_that_moved(calls, bits):
    opt, params, _ = make(bits)
    opt.step()
    expect(calls[-1], opt)
    for p in params:
        new = some(p.numel(), BF16)
        p.data = new
        opt.step()
        expect(calls[-1], opt)
        assert new.data_ptr() in [row["param"] for row in calls[-1][0]]


def test_gradients_that_moved(calls):
    opt, _, grads = make()
    grads[1].data = new = some(SIZES[1])
    opt.step()
    expect(calls[-1], opt)
    assert calls[-1][0][1]["grad"] == new.data_ptr()
    opt.grads = given = [some(n) for n in SIZES]
    opt.step()
    assert [row["grad"] for row in calls[-1][0]] == [g.data_ptr() for g in given]
    opt.grads = None
    with pytest.raises(ValueError, match="gradients"):
        opt.step()
    opt.step(given)


@pytest.mark.parametrize("bits", [8, 32])
def test_states_that_are_replaced(calls, bits):
    opt, _, _ = make(bits)
    m, v = (E4M3, E5M2) if bits == 8 else (F32, F32)
    blocks = [-(-n // 128) for n in SIZES]
    new = dict(exp_avg=[some(n, m) for n in SIZES], exp_avg_sq=[some(n, v) for n in SIZES],
               master=[some(n) for n in SIZES])
    if bits == 8:
        new.update(exp_avg_scale=[some(n) for n in blocks], exp_avg_sq_scale=[some(n) for n in blocks])
    for name, tensors in new.items():
        setattr(opt, name, tensors)
        opt.step()
        assert [row[name] for row in calls[-1][0]] == [t.data_ptr() for t in tensors]
        expect(calls[-1], opt)
    opt.steps = steps = here(torch.full((1,), 7, dtype=I64))
    opt.step()
    assert calls[-1][1] == steps.data_ptr() and opt.steps.item() == 7
    expect(calls[-1], opt)


def test_states_are_not_replaced_by_halves(calls):
    """An entry, or the storage of an alias, is no way to replace a state: the optimizer keeps its own."""
    opt, _, _ = make()
    opt.step()
    for name in ("params", "grads", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"):
        with pytest.raises(TypeError):
            getattr(opt, name)[0] = some(SIZES[0])
    with pytest.raises(AttributeError):
        opt.params = [some(n, BF16) for n in SIZES]
    mine = [some(n, E4M3) for n in SIZES]
    opt.exp_avg = mine
    at = [t.data_ptr() for t in mine]
    for t in (mine[0], opt.exp_avg[1]):
        t.data = some(t.numel(), E4M3)
    del mine, t
    opt.step()
    assert [row["exp_avg"] for row in calls[-1][0]] == at == [t.data_ptr() for t in opt.exp_avg]
    opt.exp_avg[0].copy_(torch.zeros(SIZES[0]).to(E4M3))
    assert not opt.exp_avg[0].float().any()


def test_replacements_that_do_not_fit(calls):
    """They are refused, and what was there stays."""
    opt, params, grads = make()
    opt.step()
    wrong = [("exp_avg", [some(n) for n in SIZES]), ("exp_avg", [some(n + 1, E4M3) for n in SIZES]), ("exp_avg", None),
             ("exp_avg_sq", [some(SIZES[0], E5M2)]), ("exp_avg_scale", [some(n) for n in SIZES]), ("steps", some(1)),
             ("steps", here(torch.zeros(2, dtype=I64))), ("master", [some(n, BF16) for n in SIZES]),
             ("master", [some(SIZES[0])]), ("grads", [some(n + 1) for n in SIZES]), ("grads", [some(SIZES[0])]),
             ("exp_avg", [some(2 * n, E4M3)[::2] for n in SIZES])]
    for name, tensors in wrong:
        with pytest.raises((TypeError, ValueError)):
            setattr(opt, name, tensors)
        opt.step()
        assert calls[-1] == calls[0]
    old = params[0].data
    for moved in (some(SIZES[0] + 1, BF16), some(SIZES[0], torch.float16), some(2 * SIZES[0], BF16)[::2]):
        params[0].data = moved
        count = len(calls)
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            opt.step()
        assert len(calls) == count
    params[0].data = old
    opt.step()
    expect(calls[-1], opt)


def test_memory_that_moved_is_not_taken_for_another(calls):
    """What a moved param leaves stays taken until the step that sees it: nothing else gets its address before."""
    opt, params, _ = make()
    opt.step()
    at = params[0].data_ptr()
    params[0].data = torch.zeros(0, dtype=BF16)
    others = [torch.empty(SIZES[0], dtype=BF16) for _ in range(64)]
    assert at not in [t.data_ptr() for t in others]
    params[0].data = others[0]
    opt.step()
    expect(calls[-1], opt)


def views(dtype, *ranges):
    whole = some(400, dtype)
    return [whole[a:b] for a, b in ranges]


@pytest.mark.parametrize("ranges,fine", [(((0, 40), (8, 48)), False), (((0, 40), (39, 60)), False), (((0, 40), (0, 40)), False),
                                         (((8, 16), (0, 40)), False), (((0, 40), (40, 80)), True), (((40, 80), (0, 40)), True),
                                         (((0, 40), (20, 20), (40, 80)), True)])
def test_memory_that_would_be_written_twice(calls, ranges, fine):
    """Tensors that share some memory are refused, neighbours and empty ones are not."""
    def grads():
        return [some(b - a) for a, b in ranges]

    def attempt(params, **given):
        if fine:
            dgl.AdamW(params, grads(), **given).step()
        else:
            with pytest.raises(ValueError, match="overlap"):
                dgl.AdamW(params, grads(), **given)

    def apart(dtype):
        return [some(b - a, dtype) for a, b in ranges]

    attempt(views(F32, *ranges))
    attempt(apart(BF16), master=views(F32, *ranges))
    attempt(apart(F32), exp_avg=views(F32, *ranges))
    attempt(apart(F32), exp_avg=views(E4M3, *ranges), exp_avg_sq=apart(E5M2))
    attempt(apart(F32), exp_avg=views(E4M3, *ranges), exp_avg_sq=views(E5M2, *ranges))


def test_memory_that_lists_share(calls):
    """A param that is a part of a state, of a master or of the step counter's buffer; a replacement that overlaps."""
    whole = some(400)
    for given in (dict(exp_avg=[whole[100:300]]), dict(exp_avg_sq=[whole[0:200]]), dict(steps=whole[150:152].view(I64))):
        with pytest.raises(ValueError, match="overlap"):
            dgl.AdamW([whole[:200]], [some(200)], **given)
    opt = dgl.AdamW([whole[:200]], [some(200)])
    with pytest.raises(ValueError, match="overlap"):
        opt.exp_avg = [whole[199:399]]
    with pytest.raises(ValueError, match="overlap"):
        opt.steps = opt.exp_avg[0][2:4].view(I64)
    opt.exp_avg = [whole[200:]]
    opt.step()


@pytest.mark.parametrize("how", ["of the optimizer", "of the step"])
def test_a_step_on_another_stream_is_noted(calls, monkeypatch, how):
    """Everything that the step reads or writes is marked as used on its stream, the learning rate's tensor too."""
    import contextlib
    noted = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    monkeypatch.setattr(OnDevice, "record_stream", lambda self, s: noted.append((self.data_ptr(), s)), raising=False)
    opt, params, grads = make()
    lr, scale = some(1), some(1)
    if how == "of the step":
        opt.step(lr=lr, grad_scale=scale, stream="s")
    else:
        opt.lr = lr
        opt.step(grad_scale=scale, stream="s")
    used = [*params, *grads, *opt.master, *opt.exp_avg, *opt.exp_avg_sq, *opt.exp_avg_scale, *opt.exp_avg_sq_scale, opt.steps,
            lr, scale]
    assert {(t.data_ptr(), "s") for t in used} <= set(noted)


def test_params_that_are_no_tensors(calls):
    for bad in ([3.0], ["p"], [None], [torch.nn.Linear(2, 2)], [some(8, I64)]):
        for given in (dict(), dict(master=True), dict(state_bits=8)):
            with pytest.raises(TypeError, match="params"):
                dgl.AdamW(bad, **given)
