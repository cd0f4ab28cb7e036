"""AdamW against its definition in fp64.

u is fp32's unit roundoff.  m and v take three and four roundings, each of at
most u of the sum of magnitudes; the update, lr m^ / (sqrt(v^) + eps), one of
2 u and a dozen of u; p two more of itself.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
U = 2.0**-24
B1, B2, EPS, LR = 0.9, 0.999, 1e-8, 1e-2


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


def step64(p, g, m, v, t, decay, lr=LR, b1=B1, b2=B2, eps=EPS):
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    return p * (1 - lr * decay) - lr * (m / (1 - b1**t)) / ((v / (1 - b2**t)).sqrt() + eps), m, v


def make(sizes, p_dtype, g_dtype, offset=0, seed=0):
    """Tensors that begin `offset` elements into their buffers."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def one(n, dtype, size):
        return (size * torch.randn(n + offset, device="cuda", generator=gen)).to(dtype)[offset:]

    return [one(n, p_dtype, 1.0) for n in sizes], [one(n, g_dtype, 0.01) for n in sizes]


SIZES = [1, 3, 0, 8, 127, 128, 129, 2047, 2048, 2049, 5000, 70001]


@pytest.mark.parametrize("p_dtype,g_dtype,master", [(F32, F32, False), (F32, BF16, False), (BF16, F32, True),
                                                    (BF16, BF16, True), (BF16, BF16, False)])
@pytest.mark.parametrize("offset", [0, 4, 8, 1])
def test_32_bits(dgl, p_dtype, g_dtype, master, offset):
    params, grads = make(SIZES, p_dtype, g_dtype, offset)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    opt = dgl.AdamW(params, grads, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decay, master=master or None)
    p64 = [p.double() for p in params]
    m64 = [torch.zeros_like(p) for p in p64]
    v64 = [torch.zeros_like(p) for p in p64]
    scale = torch.tensor(0.5, device="cuda")
    for t in range(1, 5):
        s = scale if t > 2 else None
        opt.step(grad_scale=s)
        assert opt.steps.item() == t and opt._ticket.item() == 0
        for i, g in enumerate(grads):
            before = p64[i]
            p64[i], m64[i], v64[i] = step64(before, g.double() * (1.0 if s is None else 0.5), m64[i], v64[i], t, decay[i])
            k = 4 * t  # roundings so far
            assert ((opt.exp_avg[i].double() - m64[i]).abs() <= k * U * 0.1).all()
            assert ((opt.exp_avg_sq[i].double() - v64[i]).abs() <= k * U * v64[i] + 1e-30).all()
            got = (opt.master[i] if master else params[i]).double()
            if p_dtype == BF16 and not master:
                tol = 2.0**-8 * p64[i].abs() * 1.01 + 1e-6  # this step's rounding
            else:
                tol = t * (3 * U * (before.abs() + LR) + 20 * U * LR)
            # near a gradient that cancels m, the update's error is m's error over sqrt(v)
            tol = tol + LR * k * U * 0.1 / (v64[i] / (1 - B2**t)).sqrt().clamp(min=1e-12)
            assert ((got - p64[i]).abs() <= tol).all()
            if master:
                assert torch.equal(params[i], opt.master[i].bfloat16())
            if p_dtype == BF16 and not master:
                p64[i] = params[i].double()
    assert dgl.device_status() == dgl.DGL_OK


def test_many_tensors(dgl):
    """More tensors than a launch holds: each is updated once, and the step counted once."""
    sizes = [(7 * i) % 300 + 1 for i in range(1000)]
    params, grads = make(sizes, F32, F32)
    start = [p.double() for p in params]
    opt = dgl.AdamW(params, lr=LR, weight_decay=0.1)
    opt.step(grads)
    assert opt.steps.item() == 1
    for p, p0, g in zip(params, start, grads):
        want, _, _ = step64(p0, g.double(), 0 * p0, 0 * p0, 1, 0.1)
        # a first step is lr times the gradient's sign
        assert ((p.double() - want).abs() <= 4 * U * (p0.abs() + LR) + 40 * U * LR + LR * EPS / g.double().abs().clamp(min=1e-9) * 1e-5).all()


def test_large_tensor(dgl):
    """Offsets past 2^31 elements, in 8-bit states."""
    n = (1 << 31) + 1000
    p = torch.zeros(n, dtype=BF16, device="cuda")
    g = torch.zeros(n, dtype=BF16, device="cuda")
    g[-1000:] = 1.0
    opt = dgl.AdamW([p], [g], lr=LR, weight_decay=0.0, state_bits=8)
    opt.step()
    assert torch.allclose(p[-1000:].float(), torch.full((1000,), -LR, device="cuda"), rtol=2.0**-8)
    assert not p[:4096].any() and not p[n // 2:n // 2 + 4096].any()
    assert not opt.exp_avg[0][:4096].view(torch.uint8).any() and opt.exp_avg[0][-1000:].view(torch.uint8).all()


def decode(codes, scale):
    n = codes.numel()
    return codes.double() * scale.double().repeat_interleave(128)[:n]


def ulp(x, scale, lowest, mantissa):
    """Distance between neighbouring codes at |x|."""
    n = x.numel()
    s = scale.double().repeat_interleave(128)[:n]
    return s * 2.0 ** (torch.floor(torch.log2((x.abs() / s).clamp(min=2.0**lowest))) - mantissa)


@pytest.mark.parametrize("p_dtype,g_dtype,master", [(F32, BF16, False), (F32, F32, False), (BF16, BF16, True)])
@pytest.mark.parametrize("offset", [0, 8, 1])
def test_8_bits(dgl, p_dtype, g_dtype, master, offset):
    """Every state is one of the two codes around its value, the block's largest sets the scale, and the
    update uses the values before they are rounded."""
    params, grads = make(SIZES, p_dtype, g_dtype, offset)
    opt = dgl.AdamW(params, grads, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=0.1, master=master or None, state_bits=8,
                    seed=5)
    for t in range(1, 5):
        old = [(decode(m, ms), decode(v, vs)) for m, ms, v, vs in
               zip(opt.exp_avg, opt.exp_avg_scale, opt.exp_avg_sq, opt.exp_avg_sq_scale)]
        before = [p.double() for p in (opt.master if master else params)]
        opt.step()
        for i, g in enumerate(grads):
            if not g.numel():
                continue
            p, m, v = step64(before[i], g.double(), *old[i], t, 0.1)
            got = (opt.master[i] if master else params[i]).double()
            tol = 3 * U * (before[i].abs() + LR) + 20 * U * LR + LR * 4 * U * 0.1 / (v / (1 - B2**t)).sqrt().clamp(min=1e-12)
            assert ((got - p).abs() <= tol).all()
            for x, codes, scale, top, lowest, mantissa in (
                    (m, opt.exp_avg[i], opt.exp_avg_scale[i], 7, -6, 3),
                    (v, opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i], 14, -14, 2)):
                blocks = torch.nn.functional.pad(x, (0, -x.numel() % 128)).view(-1, 128).abs().amax(1)
                assert (torch.log2(scale) == torch.log2(scale).round()).all()
                ratio = blocks / scale.double()
                assert ((ratio >= 2.0**top * (1 - 8 * U)) & (ratio < 2.0 ** (top + 1) * (1 + 8 * U))).all()
                far = (decode(codes, scale) - x).abs() / ulp(x, scale, lowest, mantissa)
                assert (far <= 1 + 1e-3).all()
            assert (decode(opt.exp_avg_sq[i], opt.exp_avg_sq_scale[i])[v > 0] > 0).all()


def test_8_bits_keep_their_expectation(dgl):
    """The average of a million equal values, each rounded by itself, is the value; rounded to nearest, v would
    never leave its first code."""
    n = 1 << 20
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), 0.013, device="cuda")
    opt = dgl.AdamW([p], [g], lr=0.0, betas=(0.9, 0.999), weight_decay=0.0, state_bits=8, seed=11)
    m = v = 0.0
    steps = 300
    for _ in range(steps):
        opt.step()
        m, v = 0.9 * m + 0.1 * 0.013, 0.999 * v + 0.001 * 0.013**2
    got_m = decode(opt.exp_avg[0], opt.exp_avg_scale[0]).mean().item()
    got_v = decode(opt.exp_avg_sq[0], opt.exp_avg_sq_scale[0]).mean().item()
    # an element's v wanders by at most half of itself: a million average to 5e-4 of it; a step's
    # choice is off by at most 2^-16 of a quarter of v, over 300 steps 1.2e-3 of it
    assert abs(got_v / v - 1) < 5 * 5e-4 + 1.2e-3
    assert abs(got_m / m - 1) < 5 * 2e-4 + 1e-3


def test_8_bits_by_seed(dgl):
    """Equal seeds give equal bits, others other roundings, and two steps' roundings differ."""
    def run(seed, steps=2):
        params, grads = make([5000, 300], F32, BF16)
        opt = dgl.AdamW(params, grads, lr=LR, state_bits=8, seed=seed)
        for _ in range(steps):
            opt.step()
        return [t.view(torch.uint8).clone() for t in (*opt.exp_avg, *opt.exp_avg_sq)]

    a, b, c = run(1), run(1), run(2)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert any(not torch.equal(x, y) for x, y in zip(a, c))


def test_8_bits_that_are_not_finite(dgl):
    """NaN and infinite gradients: their own element's states are NaN, the others of the block are not."""
    params, grads = make([300], F32, F32)
    clean = dgl.AdamW([params[0].clone()], [grads[0].clone()], lr=LR, state_bits=8)
    clean.step()
    grads[0][5], grads[0][140] = float("nan"), float("inf")
    opt = dgl.AdamW(params, grads, lr=LR, state_bits=8)
    opt.step()
    bad = torch.zeros(300, dtype=torch.bool, device="cuda")
    bad[5] = bad[140] = True
    for a, b in ((opt.exp_avg[0], clean.exp_avg[0]), (opt.exp_avg_sq[0], clean.exp_avg_sq[0])):
        assert torch.equal(a.float().isnan(), bad)
    assert params[0][~bad].isfinite().all() and opt.exp_avg_scale[0].isfinite().all()
    assert torch.equal(params[0][~bad], clean.params[0][~bad])


def test_extreme_gradients(dgl):
    """Scales stay normal numbers from the smallest gradients to the largest."""
    for size in (1e-38, 1e-30, 1e-18, 1e10, 1e18):
        p, g = torch.zeros(256, device="cuda"), torch.full((256,), size, device="cuda")
        opt = dgl.AdamW([p], [g], lr=LR, weight_decay=0.0, state_bits=8)
        opt.step()
        for scale in (opt.exp_avg_scale[0], opt.exp_avg_sq_scale[0]):
            assert (scale >= torch.finfo(F32).tiny).all() and scale.isfinite().all()
        m = decode(opt.exp_avg[0], opt.exp_avg_scale[0])
        if size > 1e-34:
            assert ((m / (0.1 * float(torch.tensor(size))) - 1).abs() <= 2.0**-3 * 1.001).all()
        assert p.isfinite().all()


@pytest.mark.parametrize("bits", [8, 32])
def test_no_eps(dgl, bits):
    """Without eps the step is lr m / sqrt(v) whatever the gradients' size, and nothing where there was none."""
    for size in (1.0, 1e-12, 3e-18):
        p, g = torch.zeros(300, device="cuda"), torch.full((300,), size, device="cuda")
        opt = dgl.AdamW([p], [g], lr=LR, eps=0.0, weight_decay=0.0, state_bits=bits)
        opt.step()
        # at 3e-18 v is 9e-39, where fp32 is left with 20 bits of it
        assert torch.allclose(p, torch.full_like(p, -LR), rtol=1e-5)


def test_kinds_mixed(dgl):
    """Tensors of all types, on and off their units, in one call: each as in a call of its own, in 32 bits."""
    together, alone = [], []
    for seed, (p_dtype, g_dtype, master, offset) in enumerate(
            [(F32, F32, False, 0), (BF16, F32, True, 0), (F32, BF16, False, 8), (BF16, BF16, False, 0), (BF16, BF16, True, 1),
             (F32, F32, False, 1), (BF16, F32, True, 3)]):
        params, grads = make([3000, 17], p_dtype, g_dtype, offset, seed)
        for p, g in zip(params, grads):
            m = p.float() if master else None
            together.append((p, g, m))
            alone.append((p.clone(), g.clone(), None if m is None else m.clone()))
    opt = dgl.AdamW([t[0] for t in together], [t[1] for t in together], lr=LR, master=[t[2] for t in together])
    for _ in range(3):
        opt.step()
    assert opt.steps.item() == 3
    for (p, _, m), (q, g, n) in zip(together, alone):
        one = dgl.AdamW([q], [g], lr=LR, master=[n])
        for _ in range(3):
            one.step()
        assert torch.equal(p, q) and (m is None or torch.equal(m, n))


def test_graph(dgl):
    """A captured step replayed takes the next step each time; the learning rate and the scale are read anew."""
    def fresh():
        params, grads = make([1000, 4096, 77], F32, F32)
        return params, grads, dgl.AdamW(params, grads, lr=LR, state_bits=8, seed=3)

    lrs = [0.01, 0.02, 0.005]
    lr, scale = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    want_p, _, want = fresh()
    for k, x in enumerate(lrs):
        lr.fill_(x)
        scale.fill_(1.0 / (k + 1))
        want.step(lr=lr, grad_scale=scale)
    params, grads, opt = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step(lr=lr, grad_scale=scale)
    assert opt.steps.item() == 0
    for k, x in enumerate(lrs):
        lr.fill_(x)
        scale.fill_(1.0 / (k + 1))
        graph.replay()
    assert opt.steps.item() == 3
    assert all(torch.equal(a, b) for a, b in zip(params, want_p))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(opt.exp_avg, want.exp_avg))


@pytest.mark.parametrize("bits", [8, 32])
def test_resume(dgl, bits):
    """The states, params and the number of steps are all that a run goes on from."""
    params, grads = make([900, 130], BF16, F32)
    opt = dgl.AdamW(params, grads, lr=LR, master=True, state_bits=bits, seed=7)
    opt.step()
    kept = dict(master=[t.clone() for t in opt.master], exp_avg=[t.clone() for t in opt.exp_avg],
                exp_avg_sq=[t.clone() for t in opt.exp_avg_sq], steps=opt.steps.clone(), seed=7)
    if bits == 8:
        kept.update(exp_avg_scale=[t.clone() for t in opt.exp_avg_scale],
                    exp_avg_sq_scale=[t.clone() for t in opt.exp_avg_sq_scale])
    copy = [p.clone() for p in params]
    opt.step()
    again = dgl.AdamW(copy, grads, lr=LR, **kept)
    again.step()
    assert all(torch.equal(a, b) for a, b in zip(params, copy)) and again.steps.item() == 2


def test_no_tensors_and_betas_of_zero(dgl):
    opt = dgl.AdamW([], [], lr=LR)
    opt.step()
    assert opt.steps.item() == 1
    p, g = torch.ones(10, device="cuda"), torch.full((10,), 2.0, device="cuda")
    opt = dgl.AdamW([p], [g], lr=LR, betas=(0.0, 0.0), weight_decay=0.0)
    opt.step()
    assert torch.allclose(p, torch.full_like(p, 1 - LR))
    assert math.isclose(opt.exp_avg_sq[0][0].item(), 4.0)


def test_another_stream(dgl):
    params, grads = make([50000], F32, F32)
    want = params[0].clone()
    ref = dgl.AdamW([want], [grads[0].clone()], lr=LR)
    for _ in range(3):
        ref.step()
    opt = dgl.AdamW(params, grads, lr=LR)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        opt.step(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(params[0], want)
