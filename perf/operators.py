"""The losses of a language-model head, as measured cases.

A case is one call of an operator: the cross entropy of a linear head over a
large vocabulary (``xent``) or the distillation loss against a teacher's top
logits (``distill``), each as a forward pass (``fwd``: the loss and the
log-normaliser of every token) or with its gradient (``grad``: also dX and
dW).  X [T, d] are the hidden states, W [V, d] the head's weights, both bf16.

  z = scale x . w        lse = log sum_v exp z_v        p = exp(z - lse)
  xent:     loss = lse - z_y,                  dz = g (p - onehot(y)); ignored tokens: 0
  distill:  q = softmax(teacher logits / temperature) over the kept entries,
            loss = sum_k q_k (log q_k - log p_k),  dz = g (p - q); no entry kept: 0
  dX = scale dz W,  dW = scale dz^T X           (distill: scale = 1 / temperature)
"""
import math

import torch

own = False

IGNORE = -100


def listed():
    return [
        # scoring the next token of one sequence: W is read once, latency counts
        {"name": "xent fwd 1 token", "op": "xent", "dir": "fwd", "T": 1, "V": 50257, "d": 2048},
        # perplexity of one ragged document
        {"name": "xent fwd 333", "op": "xent", "dir": "fwd", "T": 333, "V": 50257, "d": 1024},
        # perplexity of an evaluation batch at the wide model's width
        {"name": "xent fwd 4096", "op": "xent", "dir": "fwd", "T": 4096, "V": 32000, "d": 4096},
        # fine-tuning on a few tokens with a small odd vocabulary: launches count
        {"name": "xent grad 48", "op": "xent", "dir": "grad", "T": 48, "V": 4095, "d": 512},
        # the lm_head shape of the ragged GEMM sweep, as a training step
        {"name": "xent grad 1024", "op": "xent", "dir": "grad", "T": 1024, "V": 50257, "d": 512},
        # an odd packed batch at the wide model's width
        {"name": "xent grad 4095", "op": "xent", "dir": "grad", "T": 4095, "V": 32000, "d": 4096},
        # 5 x 2048 tokens of the d_model 2048 training step: the largest
        {"name": "xent grad 10240", "op": "xent", "dir": "grad", "T": 10240, "V": 50257, "d": 2048},
        # online distillation while serving: one short batch against 8 kept logits
        {"name": "distill fwd 16", "op": "distill", "dir": "fwd", "T": 16, "V": 32000, "d": 4096, "K": 8, "temp": 1.0},
        # validation of a distilled model
        {"name": "distill fwd 2047", "op": "distill", "dir": "fwd", "T": 2047, "V": 50257, "d": 1024, "K": 64, "temp": 2.0},
        # a small odd student, few kept logits
        {"name": "distill grad 131", "op": "distill", "dir": "grad", "T": 131, "V": 11007, "d": 1024, "K": 5, "temp": 1.0},
        # the lm_head shape with 64 kept logits
        {"name": "distill grad 1024", "op": "distill", "dir": "grad", "T": 1024, "V": 50257, "d": 512, "K": 64, "temp": 2.0},
        # a training batch at the wide model's width
        {"name": "distill grad 8192", "op": "distill", "dir": "grad", "T": 8192, "V": 32000, "d": 4096, "K": 32, "temp": 1.5},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    T, V, d = log_int(1, 10240), log_int(1000, 131072), 8 * log_int(8, 512)
    # no more logits, and no more work, than the largest listed case
    T = max(1, min(T, 10240 * 50257 // V, int(1.05e12 / (V * d))))
    case = {"op": rng.choice(["xent", "distill"]), "dir": rng.choice(["fwd", "grad"]), "T": T, "V": V, "d": d}
    if case["op"] == "distill":
        case["K"] = log_int(1, 128)
        case["temp"] = rng.choice([1.0, 1.5, 2.0, 4.0])
    return case


def prepare(case, seed):
    T, V, d = case["T"], case["V"], case["d"]
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    state = dict(case)
    # weights N(0, 0.02^2); hidden states N(0, 1) with a pull towards the
    # token that the row should predict, from none to a nearly certain one
    W = (0.02 * torch.randn(V, d, device="cuda", generator=gen)).bfloat16()
    X = torch.randn(T, d, device="cuda", generator=gen)
    # token frequencies fall off like 1 / rank
    top = (torch.exp(uniform(T) * math.log(V)) - 1.0).long().clamp_(0, V - 1)
    w_top = W[top].float()
    # (in a call on a few tokens to even odds: below that a loss is the small
    # difference of two logits, and 32 bits of them say little about it)
    reach = 16.0 if T > 64 else 0.8 * math.log(V)
    pull = reach * uniform(T) / w_top.square().sum(1)
    X = (X + pull[:, None] * w_top).bfloat16()
    if case["op"] == "xent":
        # every tenth token is padding or prompt; a call on a few tokens scores all of them
        target = torch.where((uniform(T) < 0.1) & (T > 16), IGNORE, top)
        live = (target != IGNORE).sum().clamp(min=1)
        state.update(target=target, g=(torch.ones(T, device="cuda") / live).float())
    else:
        K = case["K"]
        # K distinct tokens a row, the first the likeliest, logits falling off
        step = 1 + (uniform(T) * (V // K - 1)).long()
        indices = (top[:, None] + step[:, None] * torch.arange(K, device="cuda")) % V
        gaps = -torch.log(uniform(T, K).clamp_(min=1e-6)) * (8.0 / K)
        logits = 14.0 - torch.cumsum(gaps, 1)
        # rows keep from half to all of their entries (top-p), a few rows none (padding)
        kept = (K * (0.5 + 0.5 * uniform(T))).ceil() * ((uniform(T) > 0.05) | (T <= 16))
        indices = torch.where(torch.arange(K, device="cuda") < kept[:, None], indices, -1)
        live = (kept > 0).sum().clamp(min=1)
        g = torch.full((T,), case["temp"] ** 2, device="cuda") / live
        state.update(indices=indices, logits=logits.float().contiguous(), g=g.float())
    state.update(X=X.contiguous(), W=W)
    return state


def run(state):
    grad = state["dir"] == "grad"
    X, W = state["X"], state["W"]
    if own:
        import dense_gemm_linear_gb300 as dgl
        g = state["g"] if grad else None
        if state["op"] == "xent":
            return dgl.linear_cross_entropy(X, W, state["target"], g, ignore_index=IGNORE)
        return dgl.linear_distill(X, W, state["indices"], state["logits"], g, temperature=state["temp"])

    Xf, Wf = X.float(), W.float()
    scale = 1.0 if state["op"] == "xent" else 1.0 / state["temp"]
    z = scale * (Xf @ Wf.T)
    high = z.amax(1, keepdim=True)
    lse = high[:, 0] + torch.log(torch.exp(z - high).sum(1))
    if state["op"] == "xent":
        live = state["target"] != IGNORE
        at = torch.where(live, state["target"], 0)[:, None]
        loss = torch.where(live, lse - z.gather(1, at)[:, 0], 0.0)
        q = live.float()[:, None]
    else:
        kept = state["indices"] >= 0
        live = kept.any(1)
        at = torch.where(kept, state["indices"], 0)
        lq = torch.where(kept, state["logits"] * scale, -torch.inf)
        e = torch.exp(lq - torch.where(live, lq.amax(1), 0.0)[:, None])
        total = e.sum(1, keepdim=True)
        q = torch.where(live[:, None], e / total, 0.0)
        log_q = torch.where(q > 0, torch.log(q.clamp(min=1e-38)), 0.0)
        loss = (q * (log_q - (z.gather(1, at) - lse[:, None]))).sum(1)
    if not grad:
        return loss, lse
    dz = torch.exp(z - lse[:, None]) * live.float()[:, None]
    dz.scatter_add_(1, at, -q)
    dz *= (scale * state["g"])[:, None]
    return loss, lse, (dz @ Wf).bfloat16(), (dz.T @ Xf).bfloat16()


def work(case):
    T, V, d = case["T"], case["V"], case["d"]
    per_token = 8 if case["op"] == "xent" else 12 * case["K"]  # targets, or indices and teacher logits
    grad = case["dir"] == "grad"
    # X and W read, loss and lse written; with the gradient also its weights read, dX and dW written
    moved = 2 * (T + V) * d + (per_token + 8) * T + (2 * (T + V) * d + 4 * T if grad else 0)
    return {"bytes": moved, "flops": (6 if grad else 2) * T * V * d}


def exact(case, seed):
    """The definitions in 64 bits, a block of tokens at a time."""
    T, V, d = case["T"], case["V"], case["d"]
    grad = case["dir"] == "grad"
    if (6 if grad else 2) * T * V * d > 1.0e13:
        return None
    s = prepare(case, seed)
    W = s["W"].double()
    scale = 1.0 / case.get("temp", 1.0)
    losses, lses, dXs, dW = [], [], [], torch.zeros_like(W)
    rows = max(1, min(T, (1 << 28) // V))
    for t in range(0, T, rows):
        x = s["X"][t:t + rows].double()
        n = x.shape[0]
        log_p = torch.log_softmax(torch.matmul(x, W.t()) * scale, dim=1)
        lses.append(torch.logsumexp(torch.matmul(x, W.t()) * scale, dim=1))
        want = torch.zeros(n, V, dtype=torch.float64, device="cuda")  # the distribution asked for
        if case["op"] == "xent":
            r = torch.nonzero(s["target"][t:t + rows] != IGNORE)[:, 0]
            want[r, s["target"][t:t + rows][r]] = 1.0
        else:
            idx = s["indices"][t:t + rows]
            r, k = torch.nonzero(idx >= 0, as_tuple=True)
            teacher = torch.full((n, case["K"]), -math.inf, dtype=torch.float64, device="cuda")
            teacher[r, k] = s["logits"][t:t + rows][r, k].double() * scale
            want[r, idx[r, k]] = torch.softmax(teacher, 1)[r, k]
        losses.append((torch.special.xlogy(want, want) - want * log_p).sum(1))
        if grad:
            dz = (want.sum(1, keepdim=True).round() * log_p.exp() - want) * (s["g"][t:t + rows].double() * scale)[:, None]
            dXs.append(torch.matmul(dz, W))
            dW += torch.matmul(dz.t(), x)
    out = (torch.cat(losses), torch.cat(lses))
    return out + (torch.cat(dXs), dW) if grad else out
