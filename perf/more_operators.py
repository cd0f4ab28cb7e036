"""What a language model's training step needs around its linear layers and its
head, as measured cases.

  embed  fwd   Y[t] = scale W[token_t]                      (ignored tokens: zeros)
         grad  dW[v] = scale sum_{t: token_t = v} dY[t]     (into a new dW, or added to an fp32 one)
  norm   fwd   mean = mean_j x_j, rstd = 1 / sqrt(mean_j (x_j - mean)^2 + eps), y = (x - mean) rstd w + b
         grad  h = (x - mean) rstd, u = dy w:  dx = rstd (u - mean_j u - h mean_j (u h)),
               dw = sum_rows dy h,  db = sum_rows dy
  adamw        g = grad_scale grad,  m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2,
               p = p (1 - lr wd) - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
               over many tensors, m and v in 32 bits or in 8

An 8-bit state is E4M3 (m) or E5M2 (v) values times the power of two of their
block of 128 elements, rounded up or down at random so that a long average
keeps moving; the random numbers are a function of seed, step and element.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-5
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.999, 1e-8, 3e-4, 0.1
BLOCK = 128
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # the norm of one token while serving: latency counts
        {"name": "norm fwd 1 x 4096", "op": "norm", "dir": "fwd", "rows": 1, "d": 4096, "x": "bf16", "w": "fp32"},
        # 5 x 2048 tokens of the d_model 2048 training step
        {"name": "norm fwd 10240 x 2048", "op": "norm", "dir": "fwd", "rows": 10240, "d": 2048, "x": "bf16", "w": "fp32"},
        # a ragged batch of odd width, in fp32
        {"name": "norm grad 333 x 1023", "op": "norm", "dir": "grad", "rows": 333, "d": 1023, "x": "fp32", "w": "fp32"},
        # an odd packed batch at the wide model's width
        {"name": "norm grad 4095 x 4096", "op": "norm", "dir": "grad", "rows": 4095, "d": 4096, "x": "bf16", "w": "bf16"},
        # the tokens of the d_model 2048 training step
        {"name": "embed fwd 10240", "op": "embed", "dir": "fwd", "T": 10240, "V": 50257, "d": 2048, "scale": 1.0,
         "y": "bf16"},
        # fine-tuning on a few tokens with a small odd vocabulary: launches count
        {"name": "embed grad 48", "op": "embed", "dir": "grad", "T": 48, "V": 4095, "d": 512, "scale": 1.0, "y": "bf16",
         "dw": "bf16", "add": False},
        # the same training step's gradient, as a matrix of its own
        {"name": "embed grad 10240", "op": "embed", "dir": "grad", "T": 10240, "V": 50257, "d": 2048, "scale": 1.0,
         "y": "bf16", "dw": "bf16", "add": False},
        # tied with a head: added to the fp32 dW that the head's loss left
        {"name": "embed grad 8191 added", "op": "embed", "dir": "grad", "T": 8191, "V": 32000, "d": 4096, "scale": 64.0,
         "y": "bf16", "dw": "fp32", "add": True},
        # a small student: a few dozen small tensors, where launches count
        {"name": "adamw 32 small", "op": "adamw", "bits": 32, "layers": 4, "d": 192, "V": 1003, "p": "fp32", "g": "fp32",
         "master": False},
        # d_model 2048 with bf16 weights and fp32 masters: the largest
        {"name": "adamw 32 large", "op": "adamw", "bits": 32, "layers": 4, "d": 2048, "V": 50257, "p": "bf16", "g": "fp32",
         "master": True},
        # the same student with 8-bit states
        {"name": "adamw 8 small", "op": "adamw", "bits": 8, "layers": 6, "d": 256, "V": 4095, "p": "fp32", "g": "bf16",
         "master": False},
        # d_model 2048 with 8-bit states
        {"name": "adamw 8 large", "op": "adamw", "bits": 8, "layers": 4, "d": 2048, "V": 50257, "p": "fp32", "g": "bf16",
         "master": False},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "embed", "adamw"])
    if op == "norm":
        rows, d = log_int(1, 32768), log_int(8, 16384)
        if rng.random() < 0.5:
            d = -(-d // 8) * 8
        rows = max(1, min(rows, (1 << 26) // d))
        return {"op": op, "dir": rng.choice(["fwd", "grad"]), "rows": rows, "d": d, "x": rng.choice(["bf16", "fp32"]),
                "w": rng.choice(["bf16", "fp32"])}
    if op == "embed":
        T, V, d = log_int(1, 65536), log_int(500, 131072), log_int(32, 8192)
        if rng.random() < 0.7:
            d = -(-d // 8) * 8
        # no more of W, and of rows, than the largest cases hold
        V, T = max(500, min(V, (1 << 28) // d)), max(1, min(T, (1 << 27) // d))
        case = {"op": op, "dir": rng.choice(["fwd", "grad"]), "T": T, "V": V, "d": d, "scale": rng.choice([1.0, math.sqrt(d)]),
                "y": rng.choice(["bf16", "fp32"])}
        if case["dir"] == "grad":
            case["dw"], case["add"] = rng.choice([("bf16", False), ("fp32", False), ("fp32", True)])
        return case
    d = 8 * log_int(8, 256)
    p = rng.choice(["bf16", "fp32"])
    return {"op": op, "bits": rng.choice([8, 32]), "layers": log_int(1, 16) if d < 1024 else rng.randint(1, 3), "d": d,
            "V": log_int(500, 50257), "p": p, "g": rng.choice(["bf16", "fp32"]), "master": p == "bf16" and rng.random() < 0.7}


def _slots(case):
    """The tensors of a model of `layers` blocks, as (elements, decays): matrices first, then vectors, each
    in a slot of whole blocks of one flat buffer, as a trainer lays them out."""
    d, layers = case["d"], case["layers"]
    sizes = [case["V"] * d] + [n * d * d for n in (3, 1, 4, 4)] * layers
    return [(n, True) for n in sizes] + [(n, False) for n in (d, d, 3 * d, d, d, d, 4 * d, d) * layers]


def _offsets(case):
    at, offsets = 0, []
    for n, decays in _slots(case):
        offsets.append(at)
        at += -(-n // BLOCK) * BLOCK
    return offsets, at


def _mix(z):
    """SplitMix64's output function (Steele, Lea and Flood 2014) on int64 tensors."""
    z = (z ^ ((z >> 30) & 0x3FFFFFFFF)) * -0x40A7B892E31B1A47
    z = (z ^ ((z >> 27) & 0x1FFFFFFFFF)) * -0x6B2FB644ECCEEE15
    return z ^ ((z >> 31) & 0x1FFFFFFFF)


GOLDEN = -0x61C8864680B583EB


def _random16(n, seed, step):
    """Two random numbers below 2^16 for each of n elements: one 64-bit draw for two elements."""
    key = _mix(seed + step * GOLDEN)
    z = _mix(key + torch.arange(1, (n + 1) // 2 + 1, device="cuda") * GOLDEN)
    words = torch.stack([z, z >> 32], 1).reshape(-1)[:n]
    return words & 0xFFFF, (words >> 16) & 0xFFFF


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=gen)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=gen)

    state = dict(case)
    if case["op"] == "norm":
        rows, d, x_type, w_type = case["rows"], case["d"], DTYPES[case["x"]], DTYPES[case["w"]]
        # activations: rows of different sizes, a mean of their own, a few outlier channels
        x = normal(rows, d) * torch.exp(0.5 * normal(rows, 1)) + 0.3 * normal(rows, 1)
        x *= torch.where(uniform(d) < 0.01, 8.0, 1.0)
        state.update(x=x.to(x_type), w=(1 + 0.1 * normal(d)).to(w_type), b=(0.1 * normal(d)).to(w_type))
        if case["dir"] == "grad":
            xd = state["x"].double()
            mean = xd.mean(1)
            rstd = ((xd - mean[:, None]).square().mean(1) + EPS).rsqrt()
            state.update(dy=(1e-3 * normal(rows, d)).to(x_type), mean=mean.float(), rstd=rstd.float())
        return state
    if case["op"] == "embed":
        T, V, d, y_type = case["T"], case["V"], case["d"], DTYPES[case["y"]]
        # token frequencies fall off like 1 / rank, ranks spread over the vocabulary; every
        # twentieth token is padding
        rank = (torch.exp(uniform(T) * math.log(V)) - 1.0).long().clamp_(0, V - 1)
        tokens = torch.randperm(V, device="cuda", generator=gen)[rank]
        state["tokens"] = torch.where((uniform(T) < 0.05) & (T > 16), IGNORE, tokens)
        if case["dir"] == "fwd":
            state["W"] = (0.02 * normal(V, d)).to(y_type)
        else:
            state["dY"] = (1e-3 * normal(T, d)).to(y_type)
            if case["add"]:
                state["dW"] = 1e-3 * normal(V, d)
        return state

    slots, (offsets, total) = _slots(case), _offsets(case)
    # one size of gradient for each block, from element to element a spread over some orders of magnitude
    size = torch.exp(normal(total // BLOCK, 1) - 9.0) * torch.exp(normal(total // BLOCK, BLOCK))
    flat = {"p": 0.02 * normal(total), "g": (size * normal(total // BLOCK, BLOCK)).view(-1),
            "m": (0.3 * size * normal(total // BLOCK, BLOCK)).view(-1),
            "v": (size.square() * (0.5 + uniform(total // BLOCK, BLOCK))).view(-1)}
    del size
    # nothing between the tensors
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for at, (n, _) in zip(offsets, slots):
        live[at:at + n] = True
    for t in flat.values():
        t *= live
    del live
    if case["master"]:
        flat["master"] = flat["p"]
    flat["p"], flat["g"] = flat["p"].to(DTYPES[case["p"]], copy=case["master"]), flat["g"].to(DTYPES[case["g"]])
    if case["bits"] == 8:
        for key, dtype, top in (("m", torch.float8_e4m3fn, 7), ("v", torch.float8_e5m2, 14)):
            blocks = flat[key].view(-1, BLOCK)
            exponent = torch.frexp(blocks.abs().amax(1).clamp(min=2.0**-100))[1] - 1 - top
            flat[key + "_scale"] = torch.ldexp(torch.ones_like(blocks[:, 0]), exponent)
            flat[key] = (blocks / flat[key + "_scale"][:, None]).view(-1).to(dtype)
    state["flat"] = flat
    state["views"] = {key: [t[at // BLOCK:-(-(at + n) // BLOCK)] if key.endswith("_scale") else t[at:at + n]
                            for at, (n, _) in zip(offsets, slots)] for key, t in flat.items()}
    state["decayed"] = offsets[1 + 4 * case["layers"]]  # of the flat buffer, the part that decays
    state["decay"] = [DECAY if decays else 0.0 for _, decays in slots]
    state["steps"] = torch.full((1,), 999, dtype=torch.int64, device="cuda")  # taken so far
    state["grad_scale"] = 0.5 + 0.5 * uniform(1)  # from clipping by norm
    state["seed"] = seed
    return state


def _run_own(state):
    import dense_gemm_linear_gb300 as dgl
    if state["op"] == "norm":
        if state["dir"] == "fwd":
            return dgl.layer_norm(state["x"], state["w"], state["b"], eps=EPS)
        return dgl.layer_norm_grad(state["dy"], state["x"], state["mean"], state["rstd"], state["w"])
    if state["op"] == "embed":
        if state["dir"] == "fwd":
            return dgl.embedding(state["tokens"], state["W"], scale=state["scale"], ignore_index=IGNORE)
        if state["add"]:
            return dgl.embedding_grad(state["tokens"], state["dY"], state["V"], scale=state["scale"], ignore_index=IGNORE,
                                      dW=state["dW"], accumulate=True)
        out = dgl.OUT_BF16 if state["dw"] == "bf16" else dgl.OUT_F32
        return dgl.embedding_grad(state["tokens"], state["dY"], state["V"], scale=state["scale"], ignore_index=IGNORE,
                                  dw_dtype=out)
    if "optimizer" not in state:
        v = state["views"]
        state["optimizer"] = dgl.AdamW(v["p"], v["g"], lr=LR, betas=(BETA1, BETA2), eps=ADAM_EPS,
                                       weight_decay=state["decay"], master=v.get("master"), exp_avg=v["m"],
                                       exp_avg_sq=v["v"], exp_avg_scale=v.get("m_scale"),
                                       exp_avg_sq_scale=v.get("v_scale"), steps=state["steps"], seed=state["seed"])
    state["optimizer"].step(grad_scale=state["grad_scale"])
    return _updated(state)


def _updated(state):
    return {key: t for key, t in state["flat"].items() if key != "g"}


def _round_at_random(x, scale, top, mantissa, bias, r):
    """Codes of an 8-bit format, of |x| times a power of two that takes the block's largest below 2^(top + 1);
    r: random numbers below 2^16."""
    y = ((x.abs() * (1.0 / scale)[:, None]) * 2.0**(bias - 127)).view(torch.int32)  # exponents as the format has them
    shift = 23 - mantissa
    return (y + (r.int() << (shift - 16)) + (1 << (shift - 17))) >> shift


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "norm":
        x, w = state["x"].float(), state["w"].float()
        if state["dir"] == "fwd":
            mean = x.mean(1, keepdim=True)
            h = x - mean
            rstd = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
            y = h * rstd * w + state["b"].float()
            return y.to(state["x"].dtype), mean[:, 0], rstd[:, 0]
        dy, rstd = state["dy"].float(), state["rstd"][:, None]
        h = (x - state["mean"][:, None]) * rstd
        u = dy * w
        dx = rstd * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
        return dx.to(state["x"].dtype), (dy * h).sum(0), dy.sum(0)
    if state["op"] == "embed":
        live = state["tokens"] != IGNORE
        tokens = torch.where(live, state["tokens"], 0)
        if state["dir"] == "fwd":
            y = state["W"][tokens].float() * state["scale"]
            return torch.where(live[:, None], y, 0.0).to(state["W"].dtype)
        dY = torch.where(live[:, None], state["dY"].float() * state["scale"], 0.0)
        dW = state["dW"] if state["add"] else torch.zeros(state["V"], state["d"], device="cuda")
        dW.index_add_(0, tokens, dY)
        return dW if state["add"] else dW.to(DTYPES[state["dw"]])

    f, eight = state["flat"], state["bits"] == 8
    state["steps"] += 1
    t = state["steps"].double()
    g = f["g"].float() * state["grad_scale"]
    if eight:
        m = (f["m"].float().view(-1, BLOCK) * f["m_scale"][:, None]).view(-1)
        v = (f["v"].float().view(-1, BLOCK) * f["v_scale"][:, None]).view(-1)
    else:
        m, v = f["m"], f["v"]
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * (g * g)
    correct1 = -torch.expm1(t * math.log(BETA1))
    correct2 = -torch.expm1(t * math.log(BETA2))
    update = (LR / correct1).float() * m / (torch.sqrt(v) * correct2.rsqrt().float() + ADAM_EPS)
    p = f["master" if state["master"] else "p"].float()
    n = state["decayed"]
    p = torch.cat([p[:n] * (1 - LR * DECAY), p[n:]]) - update
    f["p"].copy_(p)
    if state["master"]:
        f["master"].copy_(p)
    if not eight:
        f["m"].copy_(m)
        f["v"].copy_(v)
        return _updated(state)
    r_m, r_v = _random16(m.numel(), state["seed"], state["steps"])
    for key, x, r, top, mantissa, bias in (("m", m, r_m, 7, 3, 7), ("v", v, r_v, 14, 2, 15)):
        blocks = x.view(-1, BLOCK)
        # the largest value's exponent field, held where the scale and its reciprocal are normal
        largest = (blocks.abs().amax(1).view(torch.int32) >> 23).clamp(min=16)
        f[key + "_scale"].copy_(((largest - top) << 23).view(torch.float32))
        code = _round_at_random(blocks, f[key + "_scale"], top, mantissa, bias, r.view(-1, BLOCK))
        if key == "m":
            code = code | torch.where(blocks < 0, 0x80, 0)
        else:
            code = torch.where(blocks > 0, code.clamp(min=1), 0)  # a v above zero stays above zero
        f[key].view(torch.uint8).copy_(code.view(-1))
    return _updated(state)


def _distinct(T, V):
    """How many rows of W the tokens of a case reach, on average."""
    v = torch.arange(1, V + 1, dtype=torch.float64)
    share = torch.log1p(1.0 / v) / math.log(V)
    return int((1.0 - torch.exp(-0.95 * T * share)).sum())


def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "norm":
        n, d, e = case["rows"] * case["d"], case["d"], size[case["x"]]
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * e + 2 * d * size[case["w"]] + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + d * size[case["w"]] + 8 * d + 8 * case["rows"], "flops": 14 * n}
    if case["op"] == "embed":
        T, V, d, e = case["T"], case["V"], case["d"], size[case["y"]]
        rows = _distinct(T, V)
        if case["dir"] == "fwd":
            return {"bytes": 8 * T + (rows + T) * d * e, "flops": T * d}
        # padding's gradient is not needed; dW is written whole, or its reached rows read and written
        written = 2 * rows * d * 4 if case["add"] else V * d * size[case["dw"]]
        return {"bytes": 8 * T + int(0.95 * T) * d * e + written, "flops": T * d}
    n = sum(n for n, _ in _slots(case))
    p, g = size[case["p"]], size[case["g"]]
    weights = 2 * 4 + p if case["master"] else 2 * p  # with a master, only it is read
    states = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": int(n * (weights + g + states)), "flops": 15 * n}


def exact(case, seed):
    """The definitions in 64 bits, a piece at a time."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        ys, means, rstds = [], [], []
        dw, db = (torch.zeros(case["d"], dtype=torch.float64, device="cuda") for _ in range(2))
        w = s["w"].double()
        for x, *more in zip(*(s[k].split(4096) for k in (("x", "dy", "mean", "rstd") if case["dir"] == "grad" else ("x",)))):
            x = x.double()
            if case["dir"] == "fwd":
                var, mean = torch.var_mean(x, dim=1, correction=0)
                ys.append((x - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * w + s["b"].double())
                means.append(mean)
                rstds.append(1.0 / torch.sqrt(var + EPS))
                continue
            dy, mean, rstd = (t.double() for t in more)
            h = (x - mean[:, None]) * rstd[:, None]
            u = dy * w
            ys.append(rstd[:, None] * (u - u.sum(1, keepdim=True) / case["d"]
                                       - h * torch.einsum("rd,rd->r", u, h)[:, None] / case["d"]))
            dw += torch.einsum("rd,rd->d", dy, h)
            db += dy.sum(0)
        return (torch.cat(ys), torch.cat(means), torch.cat(rstds)) if case["dir"] == "fwd" else (torch.cat(ys), dw, db)
    if case["op"] == "embed":
        kept = torch.nonzero(s["tokens"] != IGNORE)[:, 0]
        at = s["tokens"][kept]
        if case["dir"] == "fwd":
            y = torch.zeros(case["T"], case["d"], dtype=torch.float64, device="cuda")
            y[kept] = s["W"][at].double() * case["scale"]
            return y
        dW = s["dW"].double() if case["add"] else torch.zeros(case["V"], case["d"], dtype=torch.float64, device="cuda")
        for rows, i in zip(at.split(8192), kept.split(8192)):
            dW.index_put_((rows,), s["dY"][i].double() * case["scale"], accumulate=True)
        return dW

    f, total, step = s["flat"], s["flat"]["p"].numel(), 1000
    eight = case["bits"] == 8
    out = {k: torch.empty(t.shape, dtype=torch.float64, device="cuda") for k, t in f.items() if k != "g"}
    piece = 1 << 25
    if eight:
        r_m, r_v = _random16(total, seed, torch.tensor(step, device="cuda"))
    for at in range(0, total, piece):
        i = slice(at, min(at + piece, total))
        b = slice(i.start // BLOCK, i.stop // BLOCK)
        g = f["g"][i].double() * s["grad_scale"].double()
        old = {k: f[k][i].double() for k in "mv"}
        if eight:
            old = {k: (x.view(-1, BLOCK) * f[k + "_scale"][b, None].double()).view(-1) for k, x in old.items()}
        m = BETA1 * old["m"] + (1.0 - BETA1) * g
        v = BETA2 * old["v"] + (1.0 - BETA2) * g**2
        p = f["master" if case["master"] else "p"][i].double()
        keep = 1.0 - LR * DECAY * (torch.arange(i.start, i.stop, device="cuda") < s["decayed"])
        out["p"][i] = p * keep - LR * (m / (1 - BETA1**step)) / ((v / (1 - BETA2**step)).sqrt() + ADAM_EPS)
        if not eight:
            out["m"][i], out["v"][i] = m, v
            continue
        for k, x, r, top, lowest, mantissa in (("m", m, r_m, 7, -6, 3), ("v", v, r_v, 14, -14, 2)):
            x = x.view(-1, BLOCK)
            exponent = torch.frexp(x.abs().amax(1))[1].double() - 1
            scale = 2.0 ** (exponent.clamp(min=-111) - top)
            out[k + "_scale"][b] = scale
            y = x.abs() / scale[:, None]
            step_of = 2.0 ** (torch.frexp(y)[1].double() - 1).clamp(min=lowest) / 2**mantissa
            coded = torch.floor(y / step_of + (r[i].view(-1, BLOCK).double() + 0.5) / 65536) * step_of
            if k == "v":
                coded = torch.where(x > 0, coded.clamp(min=2.0**-16), coded)
            out[k][i] = (coded * torch.sign(x)).view(-1)
    if case["master"]:
        out["master"] = out["p"]
    return out
