"""The operators of a training step together, as examples/tied_lm.py runs them:
its gradients against autograd in fp64, its update against AdamW's formula, and
a captured step against an eager one."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tied_lm.py")
    spec = importlib.util.spec_from_file_location("tied_lm", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def reference(lm, tokens, target):
    """Losses and gradients in fp64, from the model's bf16 weights."""
    E, A, w1, b1, w2, b2 = leaves = [p.double().requires_grad_() for p in lm.params]

    def norm(t, w, b):
        c = t - t.mean(1, keepdim=True)
        return c * (c.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w + b

    x = norm(E[tokens] * math.sqrt(lm.width), w1, b1)
    u = x @ A.T
    y = norm(u * torch.sigmoid(u), w2, b2)
    z = y @ E.T
    loss = torch.logsumexp(z, 1) - z.gather(1, target[:, None])[:, 0]
    loss.mean().backward()
    return loss.detach(), [t.grad for t in leaves]


def difference(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


# Every tensor between the operators is bf16, off by at most 2^-9 of its values on
# average over rounding's uniform error (2^-8 / sqrt 12 each), eight of them on the
# longest way (h, x, u, a, y, dy, da, du, dx, dh): sqrt(10) 2^-8 / sqrt 12 =
# 0.0036 of a gradient's norm if nothing amplified it; a norm passes on relative errors with
# a factor near one, the head's dz is rounded once more.  Five times that.
LIMIT = 5 * 10**0.5 * 2**-8 / 12**0.5


@pytest.mark.parametrize("tokens,vocab,width", [(8, 64, 32), (304, 1003, 64), (2048, 4099, 256)])
def test_gradients(example, tokens, vocab, width):
    lm = example.TiedLM(vocab=vocab, width=width)
    gen = torch.Generator(device="cuda").manual_seed(3)
    t, target = example.batch(vocab, tokens, gen)
    loss = lm.gradients(t, target)
    want_loss, want = reference(lm, t, target)
    # a loss is off by its logits' errors, of the order of 2^-8 of a spread near one
    assert ((loss.double() - want_loss).abs() < 0.05).all()
    for got, w in zip(lm.grads, want):
        assert difference(got, w) < LIMIT


@pytest.mark.parametrize("bits", [32, 8])
def test_step(example, bits):
    """Every parameter moves by the formula's first step: lr g / (|g| + eps) and the decay."""
    lm = example.TiedLM(vocab=1003, width=64, state_bits=bits, lr=1e-2)
    t, target = example.batch(1003, 304, torch.Generator(device="cuda").manual_seed(3))
    before = [p.double() for p in lm.optimizer.params]
    start = [(m if m is not None else p).double() for m, p in zip(lm.optimizer.master, lm.params)]
    lm.step(t, target)
    norm = math.sqrt(sum(g.double().square().sum().item() for g in lm.grads))
    scale = 1.0 / max(norm, 1.0)
    for i, (p0, g) in enumerate(zip(start, lm.grads)):
        g = g.double() * scale
        want = p0 * (1 - 1e-2 * (0.01 if i < 2 else 0.0)) - 1e-2 * g / (g.abs() + 1e-8)
        got = (lm.optimizer.master[i] if lm.optimizer.master[i] is not None else lm.params[i]).double()
        # the scale and sums in fp32; where |g| is near eps its relative error moves the quotient
        assert ((got - want).abs() <= 1e-2 * 1e-4 + 1e-6 * p0.abs()).all()
        if lm.optimizer.master[i] is not None:
            assert torch.equal(lm.params[i], lm.optimizer.master[i].bfloat16())
    assert any(not torch.equal(b, p.double()) for b, p in zip(before, lm.params))
    assert lm.optimizer.steps.item() == 1


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_step(example, bits):
    """A step captured and replayed on new batches gives the bits of eager steps."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    batches = [example.batch(1003, 504, gen) for _ in range(3)]
    eager = example.TiedLM(vocab=1003, width=64, state_bits=bits)
    for b in batches:
        eager.step(*b)
    lm = example.TiedLM(vocab=1003, width=64, state_bits=bits)
    warm = example.TiedLM(vocab=1003, width=64, state_bits=bits)  # workspaces and libraries of the stream
    held = [x.clone() for x in batches[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm.step(*held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        lm.step(*held)
    for b in batches:
        for h, x in zip(held, b):
            h.copy_(x)
        graph.replay()
    torch.cuda.synchronize()
    assert lm.optimizer.steps.item() == 3
    assert all(torch.equal(a, b) for a, b in zip(lm.params, eager.params))


def test_example_runs(example):
    losses = example.train(steps=4, tokens=512, vocab=1003, width=64, state_bits=8)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)
