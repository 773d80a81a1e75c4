"""The head's loss and dropout as they are measured: cases, inputs, a plain form and the framework's calls.

The top of a drafter's training step: dropout on what the last layer adds to the residual
stream, the cross entropy of the unary logits over the whole vocabulary, its gradient into
the hidden state and (where the head is not frozen) the head, and dropout's gradient.

  ce            the loss of each position, and the logarithm of its sum of exponentials
  loss          the same with the gradients of h and, where asked, of the head
  dropout       y = residual + dropped x, the mask made from a counter
  dropout_grad  the same mask on a gradient, stored or added

`run` is their plain form in 32-bit torch operations, or the framework's calls where
`own` is true; `exact` is their definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
WORD = 0xFFFFFFFF


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # scoring one draft block of 8 against the verifier's tokens: the head is read once
        {"name": "ce_block", "op": "ce", "P": 8, "V": 151936, "D": 4096, "mul": 1.0, "cap": 0.0, "masked": 0.0},
        # the validation loss of 512 blocks of 8, capped logits
        {"name": "ce_packed", "op": "ce", "P": 4096, "V": 248320, "D": 5120, "mul": 1.0, "cap": 30.0, "masked": 0.125},
        # a smoke-sized step that trains the head too: latency alone
        {"name": "loss_tiny", "op": "loss", "P": 16, "V": 4096, "D": 256, "mul": 1.0, "cap": 0.0, "masked": 0.125,
         "head": True, "accumulate": False},
        # odd sizes, scaled and capped logits, the head's gradient added to an earlier micro-batch's
        {"name": "loss_odd", "op": "loss", "P": 1003, "V": 50021, "D": 1000, "mul": 0.8, "cap": 30.0, "masked": 0.3,
         "head": True, "accumulate": True},
        # eight draft blocks over the frozen verifier's head
        {"name": "loss_blocks", "op": "loss", "P": 64, "V": 151936, "D": 4096, "mul": 1.0, "cap": 0.0, "masked": 0.125,
         "head": False, "accumulate": False},
        # 64 requests' blocks of 8 over the largest head, frozen
        {"name": "loss_batched", "op": "loss", "P": 512, "V": 248320, "D": 5120, "mul": 1.0, "cap": 0.0,
         "masked": 0.125, "head": False, "accumulate": False},
        # the training-packed batch, 2048 blocks of 8: the anchors have no target
        {"name": "loss_packed", "op": "loss", "P": 16384, "V": 151936, "D": 4096, "mul": 1.0, "cap": 0.0,
         "masked": 0.125, "head": False, "accumulate": False},
        # 4096 positions with a head that learns
        {"name": "loss_head", "op": "loss", "P": 4096, "V": 151936, "D": 4096, "mul": 1.0, "cap": 0.0, "masked": 0.0,
         "head": True, "accumulate": False},
        # one draft block's rows: latency alone
        {"name": "dropout_block", "op": "dropout", "N": 8, "D": 4096, "x": "bf16", "out": "bf16", "rate": 0.1,
         "residual": True, "pad": 0, "on_gpu": False},
        # the training-packed batch's residual stream, the step's number on the GPU
        {"name": "dropout_packed", "op": "dropout", "N": 16384, "D": 5120, "x": "bf16", "out": "bf16", "rate": 0.1,
         "residual": True, "pad": 0, "on_gpu": True},
        # rows of an odd length that are further apart than they are long
        {"name": "dropout_odd", "op": "dropout", "N": 5003, "D": 251, "x": "f32", "out": "f32", "rate": 0.3,
         "residual": False, "pad": 6, "on_gpu": False},
        # the packed batch's gradient through the mask, added in 32 bits to what came by other ways
        {"name": "dropout_grad_packed", "op": "dropout_grad", "N": 16384, "D": 4096, "x": "bf16", "out": "f32",
         "rate": 0.1, "residual": True, "pad": 0, "on_gpu": False},
    ]


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce", "loss", "loss", "dropout", "dropout_grad"])
    if op in ("ce", "loss"):
        D = 8 * log_int(rng, 8, 640)
        V = log_int(rng, 1000, 248320)
        P = log_int(rng, 8, min(16384, 2 * 10 ** 12 // (V * D)))
        c = {"op": op, "P": P, "V": V, "D": D, "mul": rng.choice([1.0, 1.0, 0.8]), "cap": rng.choice([0.0, 0.0, 30.0]),
             "masked": rng.choice([0.0, 0.125, 0.5])}
        if op == "loss":
            c["head"] = rng.random() < 0.5
            c["accumulate"] = c["head"] and rng.random() < 0.5
        return c
    D = log_int(rng, 1, 5120)
    N = log_int(rng, 1, min(131072, 16384 * 5120 // D))
    return {"op": op, "N": N, "D": D, "x": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]),
            "rate": rng.choice([0.0, 0.05, 0.1, 0.5]), "residual": rng.random() < 0.5, "pad": rng.choice([0, 0, 1, 8]),
            "on_gpu": rng.random() < 0.5}


# ----------------------------------------------------------------- inputs --

def normal(gen, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    return x.to(dtype)


def uniform(gen, *shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(0.0, 1.0, generator=gen)


def rows_apart(x, pad):
    """x with `pad` elements of something else behind every row."""
    if not pad:
        return x
    wide = torch.full((x.shape[0], x.shape[1] + pad), 7.0, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("ce", "loss"):
        P, V, D = case["P"], case["V"], case["D"]
        # tokens whose frequency falls off as 1/rank; normal logits of deviation 2.5, the
        # target's raised by 0 to 12: from a guess to near certainty
        rank = torch.exp(uniform(gen, P).double() * math.log(V)).long().clamp_(1, V) - 1
        step = next(q for q in (7919, 104729, 15485863, 1) if math.gcd(q, V) == 1)
        targets = (rank * step + 11) % V
        s["W"] = normal(gen, (V, D), torch.bfloat16, 2.5 / math.sqrt(D))
        raised = uniform(gen, P, 1) * (12.0 / 6.25)
        s["h"] = (normal(gen, (P, D), torch.float32) + raised * s["W"][targets].float()).to(torch.bfloat16)
        s["targets"] = torch.where(uniform(gen, P) < case["masked"], torch.full_like(targets, -1),
                                   targets).to(torch.int32)
        if case["op"] == "loss":
            s["row_weights"] = uniform(gen, P) * (2.0 / P)
            if case["head"]:
                s["dW"] = (normal(gen, (V, D), torch.bfloat16, 1e-4) if case["accumulate"] else
                           torch.empty((V, D), dtype=torch.bfloat16, device="cuda"))
        return s
    N, D = case["N"], case["D"]
    s["x"] = rows_apart(normal(gen, (N, D), DTYPES[case["x"]]), case["pad"])
    if case["residual"]:
        s["res"] = rows_apart(normal(gen, (N, D), DTYPES[case["out"]]), case["pad"])
    s["seed"] = (seed * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 63)
    s["draw"] = (seed * 77777 + 5) % (1 << 40)
    if case["on_gpu"]:
        s["draw"] = torch.full((1,), s["draw"], dtype=torch.int64, device="cuda")
    return s


# ------------------------------------------------------------- plain form --

def plain_loss(s):
    c = s["case"]
    h, W = s["h"].float(), s["W"].float()
    live = s["targets"] >= 0
    t = s["targets"].clamp(min=0).long()[:, None]
    x = h @ W.t()
    slope = c["mul"]
    if c["mul"] != 1.0:
        x = x * c["mul"]
    if c["cap"]:
        bent = torch.tanh(x / c["cap"])
        x = bent * c["cap"]
        slope = c["mul"] * (1.0 - bent * bent)
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    xt = x.gather(1, t)
    others = e.scatter(1, t, 0.0).sum(1, keepdim=True)
    # log(others + exp(xt - top)), also where the target's share is all but one
    loss = ((top - xt) + torch.log1p(others + torch.expm1(xt - top)))[:, 0]
    lse = (top + total.log())[:, 0]
    nan = torch.full_like(loss, float("nan"))
    out = {"loss": torch.where(live, loss, nan), "lse": torch.where(live, lse, nan)}
    if c["op"] == "ce":
        return out
    # e becomes the gradient of the logits; the target's is minus the others' share
    g = e / total
    g.scatter_(1, t, -others / total)
    g = g * slope * torch.where(live, s["row_weights"], torch.zeros_like(loss))[:, None]
    out["dh"] = (g @ W).to(torch.bfloat16)
    if c["head"]:
        dW = g.t() @ h
        s["dW"].copy_(s["dW"].float() + dW if c["accumulate"] else dW)
        out["dW"] = s["dW"]
    return out


def random_words(n, seed, draw):
    """n 16-bit words: Philox4x32 of 10 rounds (Salmon et al., "Parallel random numbers: as easy as
    1, 2, 3", 2011) with the seed as its key and (number of the group of 8, draw) as its counter."""
    q = torch.arange(-(-n // 8), device="cuda", dtype=torch.int64)
    c = [q & WORD, q >> 32, draw & WORD, (draw >> 32) & WORD]
    k = [seed & WORD, (seed >> 32) & WORD]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57      # the low 64 bits, whatever their sign
        c = [((b >> 32) & WORD) ^ c[1] ^ k[0], b & WORD, ((a >> 32) & WORD) ^ c[3] ^ k[1], a & WORD]
        k = [(k[0] + 0x9E3779B9) & WORD, (k[1] + 0xBB67AE85) & WORD]
    return torch.stack([w for x in c for w in (x & 0xFFFF, x >> 16)], dim=1).view(-1)[:n]


def plain_dropout(s):
    c = s["case"]
    N, D = c["N"], c["D"]
    drop = math.floor(c["rate"] * 65536 + 0.5)
    keep = (random_words(N * D, s["seed"], s["draw"]) >= drop).view(N, D)
    y = torch.where(keep, s["x"].float() * (65536.0 / (65536 - drop)), torch.zeros((), device="cuda"))
    if c["residual"]:
        y = y + s["res"].float()
    y = y.to(DTYPES[c["out"]])
    if c["op"] == "dropout_grad" and c["residual"]:
        s["res"].copy_(y)
        return s["res"]
    return y


# -------------------------------------------------------------------- run --

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return plain_loss(s) if op in ("ce", "loss") else plain_dropout(s)
    import dflash2_draft_block_gb300 as df2
    if op == "ce":
        loss, lse = df2.unary_ce(s["h"], s["W"], s["targets"], output_multiplier=c["mul"],
                                 final_logit_softcapping=c["cap"])
        return {"loss": loss, "lse": lse}
    if op == "loss":
        loss, lse, dh, dW = df2.unary_loss_grad(
            s["h"], s["W"], s["targets"], row_weights=s["row_weights"], output_multiplier=c["mul"],
            final_logit_softcapping=c["cap"], accumulate=c["accumulate"], dW=s.get("dW"))
        out = {"loss": loss, "lse": lse, "dh": dh}
        return {**out, "dW": dW} if c["head"] else out
    if op == "dropout":
        return df2.dropout(s["x"], c["rate"], s["seed"], s["draw"], residual=s.get("res"), dtype=DTYPES[c["out"]])
    return df2.dropout_grad(s["x"], c["rate"], s["seed"], s["draw"], dtype=DTYPES[c["out"]],
                            accumulate=c["residual"], out=s.get("res"))


# ------------------------------------------------------------------- work --

def work(case):
    if case["op"] in ("ce", "loss"):
        P, V, D = case["P"], case["V"], case["D"]
        live = P * (1.0 - case["masked"])
        cost = {"bytes": 2 * (live + V) * D + 12 * P, "flops": 2 * live * V * D}
        if case["op"] == "loss":
            cost["bytes"] += 4 * P + 2 * P * D + (V * D * (4 if case["accumulate"] else 2) if case["head"] else 0)
            cost["flops"] *= 3 if case["head"] else 2
        return cost
    n = case["N"] * case["D"]
    out = SIZES[case["out"]]
    return {"bytes": n * (SIZES[case["x"]] + out * (2 if case["residual"] else 1)), "flops": 2 * n}


# ------------------------------------------------------------------ exact --

def exact_loss(case, s):
    P, V, D = case["P"], case["V"], case["D"]
    if work(case)["flops"] > 1.6e13:      # 64-bit products run at about 1e12 a second
        return None
    h, W, t = s["h"].double(), s["W"].double(), s["targets"].long()
    m, cap = case["mul"], case["cap"]
    loss = torch.full((P,), float("nan"), dtype=torch.float64, device="cuda")
    lse = loss.clone()
    grads = case["op"] == "loss"
    dh = torch.zeros((P, D), dtype=torch.float64, device="cuda") if grads else None
    dW = None
    if grads and case["head"]:
        dW = s["dW"].double() if case["accumulate"] else torch.zeros((V, D), dtype=torch.float64, device="cuda")
    for some in (t >= 0).nonzero()[:, 0].split(max(1, 2 ** 28 // V)):
        x = torch.mm(h[some], W.T) * m
        if cap:
            x = cap * torch.tanh(x / cap)
        lse[some] = torch.logsumexp(x, 1)
        loss[some] = lse[some] - x[torch.arange(len(some), device="cuda"), t[some]]
        if grads:
            g = torch.softmax(x, 1)
            g[torch.arange(len(some), device="cuda"), t[some]] = torch.expm1(-loss[some])
            g *= m * s["row_weights"].double()[some][:, None]
            if cap:
                g *= 1.0 - (x / cap) ** 2
            dh[some] = torch.mm(g, W)
            if dW is not None:
                dW += torch.mm(g.T, h[some])
    out = {"loss": loss, "lse": lse}
    if grads:
        out["dh"] = dh
        if dW is not None:
            out["dW"] = dW
    return out


def exact_words(n, seed, draw):
    """random_words in halves of 16 bits, so that no product passes 2^32."""
    def product(x, m):
        m0, m1, x0, x1 = m & 0xFFFF, m >> 16, x & 0xFFFF, x >> 16
        mid = x1 * m0 + (x0 * m0 >> 16)
        low = x0 * m1 + (mid & 0xFFFF)
        return x1 * m1 + (mid >> 16) + (low >> 16), ((low & 0xFFFF) << 16) | (x0 * m0 & 0xFFFF)

    group = torch.arange((n + 7) // 8, device="cuda")
    zero = torch.zeros_like(group)
    a, b, c, d = group % 2 ** 32, group // 2 ** 32, zero + draw % 2 ** 32, zero + draw // 2 ** 32
    for r in range(10):
        hi0, lo0 = product(a, 0xD2511F53)
        hi1, lo1 = product(c, 0xCD9E8D57)
        a, c = hi1 ^ b ^ (seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, hi0 ^ d ^ (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
        b, d = lo1, lo0
    words = torch.empty((len(group), 4, 2), dtype=torch.int32, device="cuda")
    for j, w in enumerate((a, b, c, d)):
        words[:, j, 0], words[:, j, 1] = w % 65536, w // 65536
    return words.flatten()[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ce", "loss"):
        return exact_loss(case, s)
    N, D = case["N"], case["D"]
    drawn = int(s["draw"])
    dropped = exact_words(N * D, s["seed"], drawn).reshape(N, D) < int(np.floor(case["rate"] * 65536 + 0.5))
    y = s["x"].double() / (1.0 - np.floor(case["rate"] * 65536 + 0.5) / 65536)
    y[dropped] = 0.0
    return y + s["res"].double() if case["residual"] else y
