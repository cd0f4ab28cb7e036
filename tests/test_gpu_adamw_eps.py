"""AdamW's first step, lr g / (|g| + eps), where eps, the gradients or their squares are small."""
import pytest
import torch

pytestmark = pytest.mark.gpu

LR = 1e-2


@pytest.fixture(scope="module")
def dgl():
    import dense_gemm_linear_gb300 as d
    d.load_library()
    return d


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("eps", [0.0, 2e-18, 1e-17, 1e-15, 1e-12, 1e-10, 1e-8])
@pytest.mark.parametrize("beta2", [0.999, 0.999999])
def test_first_step(dgl, bits, eps, beta2):
    for size in (1e-20, 3.3e-18, 1e-15, 1e-12, 1e-7, 1.0):
        p, g = torch.zeros(300, device="cuda"), torch.full((300,), size, device="cuda")
        opt = dgl.AdamW([p], [g], lr=LR, betas=(0.9, beta2), eps=eps, weight_decay=0.0, state_bits=bits)
        opt.step()
        g64 = g.double()
        want = -LR * g64 / (g64 + eps)
        # a few units of 2^-24 for the root, its correction and the quotient: 1e-5 holds them many times.  Where g^2 and
        # v = (1 - beta2) g^2 are subnormal, each loses up to 2^-150; half of what that is of v reaches the root
        lost = 2.0**-150 * (1 + 1 / (1 - beta2)) / size**2
        if lost > 0.25:  # nothing may be left of v: the quotient is then m / eps, off by a factor 1 + size / eps
            if eps < 100 * size:
                continue
            lost = 1.02
        tol = 1e-5 + lost * size / (size + eps)
        assert ((p.double() - want).abs() <= tol * want.abs()).all(), (size, p[0].item(), want[0].item())
