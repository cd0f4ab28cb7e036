"""The 8-bit states of AdamW bit for bit: the codes and scales computed anew from the values before the step, the seed, the
step and each element's place among the call's tensors."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
B1, B2 = 0.9, 0.999
KINDS = [(F32, F32, False, 0), (BF16, F32, True, 0), (F32, BF16, False, 8), (BF16, BF16, False, 0), (BF16, BF16, True, 1),
         (F32, F32, False, 1), (BF16, F32, True, 3)]  # param, gradient, master, elements before the tensors' first


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


def mix(z):
    """SplitMix64's output function (Steele, Lea and Flood 2014) on int64 tensors."""
    z = (z ^ ((z >> 30) & 0x3FFFFFFFF)) * -0x40A7B892E31B1A47
    z = (z ^ ((z >> 27) & 0x1FFFFFFFFF)) * -0x6B2FB644ECCEEE15
    return z ^ ((z >> 31) & 0x1FFFFFFFF)


GOLDEN = -0x61C8864680B583EB


def codes(x, random, top, mantissa, bias):
    """Codes and scales of values in blocks of 128; random: numbers below 2^16."""
    x = x.view(-1, 128)
    largest = (x.abs().amax(1).view(torch.int32) >> 23).clamp(min=16)
    scale = ((largest - top) << 23).view(F32)
    shift = 23 - mantissa
    y = (x.abs() * (1.0 / scale)[:, None] * 2.0**(bias - 127)).view(torch.int32)
    code = (y + (random.view_as(x).int() << (shift - 16)) + (1 << (shift - 17))) >> shift
    if mantissa == 3:
        code = code | torch.where(x < 0, 0x80, 0)
    else:
        code = torch.where(x > 0, code.clamp(min=1), 0)
    return code.to(torch.uint8).view(-1), scale


class Flat:
    """A list of tensors as one padded to whole blocks each, in the order of the call."""

    def __init__(self, sizes):
        self.sizes, self.at, n = sizes, [], 0
        for k in sizes:
            self.at.append(n)
            n += -(-k // 128) * 128
        self.n = n

    def join(self, tensors, dtype=F32):
        whole = torch.zeros(self.n, dtype=dtype, device="cuda")
        for t, at in zip(tensors, self.at):
            whole[at:at + t.numel()] = t.view(dtype) if dtype == torch.uint8 else t.float()
        return whole

    def scales(self, tensors):
        return torch.cat([t for t in tensors if t.numel()])


@pytest.mark.parametrize("sizes", [[5000, 0, 1, 129, 2048, 130, 127], [(37 * i) % 400 for i in range(800)]],
                         ids=["few", "more than a launch holds"])
@pytest.mark.parametrize("seed", [0, 2**63 + 12345])
def test_codes(dgl, sizes, seed):
    gen = torch.Generator(device="cuda").manual_seed(7)

    def some(n, dtype, before):
        return torch.randn(n + before, device="cuda", generator=gen).to(dtype)[before:]

    kinds = [KINDS[i % len(KINDS)] for i in range(len(sizes))]
    params = [some(n, p, before) for n, (p, _, _, before) in zip(sizes, kinds)]
    grads = [some(n, g, before) * 10.0 ** (i % 9 - 4) for i, (n, (_, g, _, before)) in enumerate(zip(sizes, kinds))]
    master = [p.float() if k[2] else None for p, k in zip(params, kinds)]
    flat = Flat(sizes)
    g = flat.join(grads)
    opt = dgl.AdamW(params, grads, betas=(B1, B2), master=master, state_bits=8, seed=seed)
    for t in range(1, 4):
        m, v = (flat.join([s.float() for s in states]).view(-1, 128) * flat.scales(scales)[:, None]
                for states, scales in ((opt.exp_avg, opt.exp_avg_scale), (opt.exp_avg_sq, opt.exp_avg_sq_scale)))
        opt.step()
        m = B1 * m.view(-1) + (1 - B1) * g
        v = B2 * v.view(-1) + (1 - B2) * (g * g)
        step = (seed + t * GOLDEN + 2**63) % 2**64 - 2**63
        z = mix(mix(torch.tensor(step, device="cuda")) + torch.arange(1, flat.n // 2 + 1, device="cuda") * GOLDEN)
        words = torch.stack([z, z >> 32], 1).reshape(-1)
        for x, random, states, scales, format in (
                (m, words & 0xFFFF, opt.exp_avg, opt.exp_avg_scale, (7, 3, 7)),
                (v, (words >> 16) & 0xFFFF, opt.exp_avg_sq, opt.exp_avg_sq_scale, (14, 2, 15))):
            code, scale = codes(x, random, *format)
            assert torch.equal(flat.scales(scales), scale)
            have = flat.join([s.view(torch.uint8) for s in states], torch.uint8)
            real = flat.join([torch.ones(k, device="cuda") for k in sizes]).bool()
            assert torch.equal(have[real], code[real])
    assert opt.steps.item() == 3


def test_places_and_steps_round_differently(dgl):
    """Equal tensors of one call, in one kind or two, and equal states a step apart."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    p, g = torch.randn(4096, device="cuda", generator=gen), torch.randn(4096, device="cuda", generator=gen)

    def step(count, steps):
        params = [torch.cat([p[:i % 2], p])[i % 2:] for i in range(count)]  # every second one off its units
        opt = dgl.AdamW(params, [g] * count, state_bits=8, seed=1,
                        steps=torch.full((1,), steps, dtype=torch.int64, device="cuda"))
        opt.step()
        return [[t.view(torch.uint8) for t in states] for states in (opt.exp_avg, opt.exp_avg_sq)]

    now, later = step(4, 0), step(1, 1)
    for a, b in zip(now, later):
        rounded = [*a, *b]
        for i in range(len(rounded)):
            for j in range(i):
                differing = (rounded[i] != rounded[j]).float().mean().item()
                assert differing > 0.1  # of codes between which both are possible, about a third differ
