#!/usr/bin/env python3
"""Trains a small student head on tokens and on a teacher's top logits.

The student is one linear layer and a head: h = SiLU(F A^T), z = h W^T, with F
the features of a batch of tokens.  A step runs, through the library alone,

  dgl.linear                 h, the layer's fused forward
  dgl.linear_cross_entropy   the loss on the tokens, dh and dW (fp32)
  dgl.linear_distill         the loss on the teacher's logits, dh, and its dW
                             added to the same buffer (accumulate)
  dgl.dgl_gemm_bf16_ex       dA = dz^T F, from dh and the activation's derivative

and applies plain SGD.  The teacher is a fixed random layer and head; its
top logits come from a full product, as a server would have stored them.

  python examples/distill_head.py [--steps 60]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_gemm_linear_gb300 as dgl  # noqa: E402


def hidden(F, A):
    """h = SiLU(F A^T) and its derivative's ingredients."""
    h = dgl.linear(F, A, act=dgl.ACT_SILU)
    pre = dgl.gemm_bf16(F, A).float()  # the backward pass needs the pre-activation
    return h, pre


def train(steps=60, tokens=512, vocab=4099, width=256, features=192, keep=16, temperature=2.0, seed=0):
    """Returns the two losses of every step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std):
        return std * torch.randn(*shape, device="cuda", generator=gen)

    teacher_A, teacher_W = normal(width, features, std=features**-0.5).bfloat16(), normal(vocab, width, std=0.4).bfloat16()
    A, W = normal(width, features, std=features**-0.5), normal(vocab, width, std=0.02)  # fp32 masters
    # a mean over the tokens; temperature^2 keeps the soft loss's gradient in step
    g_hard = torch.full((tokens,), 0.5 / tokens, device="cuda")
    g_soft = torch.full((tokens,), 0.5 * temperature**2 / tokens, device="cuda")
    dW = torch.empty(vocab, width, device="cuda")
    dA = torch.empty(width, features, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    history = []
    F = normal(tokens, features, std=1.0).bfloat16()
    t_logits = dgl.gemm_bf16(dgl.linear(F, teacher_A, act=dgl.ACT_SILU), teacher_W, out_dtype=dgl.OUT_F32)
    top, indices = t_logits.topk(keep, dim=1)
    target = indices[:, 0].contiguous()
    for _ in range(steps):
        Ab, Wb = A.bfloat16(), W.bfloat16()
        h, pre = hidden(F, Ab)
        hard, _, dh1, _ = dgl.linear_cross_entropy(h, Wb, target, g_hard, dW=dW)
        soft, _, dh2, _ = dgl.linear_distill(h, Wb, indices, top, g_soft, temperature=temperature, dW=dW,
                                             accumulate=True)
        s = torch.sigmoid(pre)
        dz = ((dh1.float() + dh2.float()) * (s * (1 + pre * (1 - s)))).bfloat16()
        st = dgl.dgl_gemm_bf16_ex(dgl.MN_MAJOR, dgl.MN_MAJOR, dz.data_ptr(), width, F.data_ptr(), features,
                                  dA.data_ptr(), features, width, features, tokens, dgl.OUT_F32, None, stream)
        if st != dgl.DGL_OK:
            raise dgl.DglError(st, "dgl_gemm_bf16_ex")
        W -= 40.0 * dW
        A -= 4.0 * dA
        history.append((hard.mean(), soft.mean()))
    if dgl.device_status() != dgl.DGL_OK:
        raise RuntimeError("a kernel gave up waiting")
    return [(a.item(), b.item()) for a, b in history]


if __name__ == "__main__":
    args = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    args.add_argument("--steps", type=int, default=60)
    losses = train(args.parse_args().steps)
    for i in sorted({0, len(losses) // 4, len(losses) // 2, len(losses) - 1}):
        print("step %4d   cross entropy %.4f   distillation %.4f" % ((i,) + losses[i]))
