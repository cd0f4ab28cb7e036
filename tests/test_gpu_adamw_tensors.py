"""AdamW whose tensors are replaced between two steps: the results of an optimizer made of the new ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
SIZES = [5000, 130, 1]


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


def make(dgl, bits, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    params = [torch.randn(n, device="cuda", generator=gen).to(BF16) for n in SIZES]
    grads = [torch.randn(n, device="cuda", generator=gen) for n in SIZES]
    return dgl.AdamW(params, grads, master=True, state_bits=bits, seed=3), params, grads


def state(opt):
    names = ["master", "exp_avg", "exp_avg_sq"] + (["exp_avg_scale", "exp_avg_sq_scale"] if opt.state_bits == 8 else [])
    return {name: [t.clone() for t in getattr(opt, name)] for name in names}


def equal(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("bits", [8, 32])
def test_checkpoint_into_a_living_optimizer(dgl, bits):
    """Its state, masters, steps and params replaced by those kept two steps before, it takes the same steps again."""
    opt, params, _ = make(dgl, bits)
    opt.step()
    kept, kept_params, steps = state(opt), [p.clone() for p in params], opt.steps.clone()
    for _ in range(2):
        opt.step()
    want, want_params = state(opt), [p.clone() for p in params]
    for name, tensors in kept.items():
        setattr(opt, name, tensors)
    opt.steps = steps
    for p, new in zip(params, kept_params):
        p.data = new
    held = [torch.full((n,), 7.0, device="cuda") for n in SIZES * 8]  # takes what memory was let go
    for _ in range(2):
        opt.step()
    assert opt.steps.item() == 3 and steps.item() == 3
    assert equal(params, want_params) and all(equal(want[name], getattr(opt, name)) for name in want)
    assert all((t == 7.0).all() for t in held)


@pytest.mark.parametrize("bits", [8, 32])
def test_params_and_gradients_that_move(dgl, bits):
    """To the host and back between steps, as a module's cpu() and cuda() do."""
    still, want, _ = make(dgl, bits)
    opt, params, grads = make(dgl, bits)
    for _ in range(3):
        still.step()
        opt.step()
        for t in (*params, *grads):
            t.data = t.data.cpu()
        with pytest.raises((TypeError, ValueError)):
            opt.step()
        between = [torch.zeros(n, device="cuda") for n in SIZES * 8]
        for t in (*params, *grads):
            t.data = t.data.cuda()
        opt.step()
        still.step()
        assert all(not t.any() for t in between)
        assert equal(params, want) and equal(opt.exp_avg, still.exp_avg)
    assert opt.steps.item() == still.steps.item() == 6
