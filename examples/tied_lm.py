#!/usr/bin/env python3
"""Trains a small language model whose head has the embedding's weights.

  h = E[tokens] sqrt(d),  x = norm(h),  u = x A^T,  a = SiLU(u),  y = norm(a)
  loss = mean of the cross entropies of y E^T

A step runs, through the library alone but for the activation,

  dgl.embedding               h
  dgl.layer_norm              x and y, with the statistics their gradients read
  dgl.gemm_bf16               u
  dgl.linear_cross_entropy    the losses, dy, and dE in fp32
  dgl.layer_norm_grad         da and dh, with the norms' weights' gradients
  dgl.dgl_gemm_bf16_ex        dx = du A and dA = du^T x
  dgl.embedding_grad          added to the dE that the head's loss left
  dgl.AdamW                   a launch for each kind of tensors

The tokens follow one another by a fixed random rule, which the model learns.

  python examples/tied_lm.py [--steps 60] [--state-bits 8]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_gemm_linear_gb300 as dgl  # noqa: E402


class TiedLM:
    """Weights in bf16 with fp32 masters, norms in fp32, and buffers for all gradients."""

    def __init__(self, vocab=4099, width=256, seed=0, state_bits=32, lr=3e-3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.width = vocab, width
        self.E = (0.02 * torch.randn(vocab, width, device="cuda", generator=gen)).bfloat16()
        self.A = (width**-0.5 * torch.randn(width, width, device="cuda", generator=gen)).bfloat16()
        ones, zeros = torch.ones(width, device="cuda"), torch.zeros(width, device="cuda")
        self.norms = [ones.clone(), zeros.clone(), ones.clone(), zeros.clone()]  # weight, bias, weight, bias
        self.params = [self.E, self.A, *self.norms]
        self.grads = [torch.empty(p.shape, device="cuda") for p in self.params]
        self.optimizer = dgl.AdamW(self.params, self.grads, lr=lr, weight_decay=[0.01, 0.01, 0.0, 0.0, 0.0, 0.0],
                                   master=True, state_bits=state_bits, seed=seed)

    def gradients(self, tokens, target):
        """The losses; the gradients of their mean go to self.grads.  The tokens are a multiple of 8: dA sums over
        them, in units of 16 bytes."""
        T, d = tokens.shape[0], self.width
        dE, dA, dw1, db1, dw2, db2 = self.grads
        w1, b1, w2, b2 = self.norms
        scale = math.sqrt(d)
        h = dgl.embedding(tokens, self.E, scale=scale)
        x, mean1, rstd1 = dgl.layer_norm(h, w1, b1)
        u = dgl.gemm_bf16(x, self.A)
        s = torch.sigmoid(u.float())
        a = (u.float() * s).bfloat16()
        y, mean2, rstd2 = dgl.layer_norm(a, w2, b2)
        g = torch.full((T,), 1.0 / T, device="cuda")
        loss, _, dy, _ = dgl.linear_cross_entropy(y, self.E, target, g, dW=dE)
        da, _, _ = dgl.layer_norm_grad(dy, a, mean2, rstd2, w2, dweight=dw2, dbias=db2)
        du = (da.float() * (s * (1 + u.float() * (1 - s)))).bfloat16()
        dx = torch.empty_like(x)
        stream = torch.cuda.current_stream().cuda_stream
        for st in (dgl.dgl_gemm_bf16_ex(dgl.K_MAJOR, dgl.MN_MAJOR, du.data_ptr(), d, self.A.data_ptr(), d, dx.data_ptr(), d,
                                        T, d, d, dgl.OUT_BF16, None, stream),
                   dgl.dgl_gemm_bf16_ex(dgl.MN_MAJOR, dgl.MN_MAJOR, du.data_ptr(), d, x.data_ptr(), d, dA.data_ptr(), d,
                                        d, d, T, dgl.OUT_F32, None, stream)):
            if st != dgl.DGL_OK:
                raise dgl.DglError(st, "dgl_gemm_bf16_ex")
        dh, _, _ = dgl.layer_norm_grad(dx, h, mean1, rstd1, w1, dweight=dw1, dbias=db1)
        dgl.embedding_grad(tokens, dh, self.vocab, scale=scale, dW=dE, accumulate=True)
        return loss

    def step(self, tokens, target):
        """A training step, with the gradients' common norm clipped to 1; returns the losses."""
        loss = self.gradients(tokens, target)
        norm = torch.stack([g.square().sum() for g in self.grads]).sum().sqrt()
        self.optimizer.step(grad_scale=(1.0 / norm.clamp(min=1.0)).view(1))
        return loss


def batch(vocab, tokens, generator):
    """Tokens and the ones that follow them."""
    t = torch.randint(0, vocab, (tokens,), device="cuda", generator=generator)
    return t, (t * 31 + 7) % vocab


def train(steps=60, tokens=2048, **model):
    """Returns the mean loss of every step."""
    lm = TiedLM(**model)
    gen = torch.Generator(device="cuda").manual_seed(1)
    history = [lm.step(*batch(lm.vocab, tokens, gen)).mean() for _ in range(steps)]
    if dgl.device_status() != dgl.DGL_OK:
        raise RuntimeError("a kernel gave up waiting")
    return [x.item() for x in history]


if __name__ == "__main__":
    args = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    args.add_argument("--steps", type=int, default=60)
    args.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    args = args.parse_args()
    losses = train(args.steps, state_bits=args.state_bits)
    for i in sorted({0, len(losses) // 4, len(losses) // 2, len(losses) - 1}):
        print("step %4d   cross entropy %.4f" % (i, losses[i]))
