"""The training operators as they are measured: cases, inputs, a plain form and the framework's calls.

The selector's training step reads embeddings by token id, takes the K-way loss of the
teacher-forced scores with its gradients, folds per-token contributions into table
gradients, and steps the weights.  Four operators:

  embed       rows of a table by token id, scaled
  embed_grad  the table's gradient from the rows' gradients
  selector    the selector's loss with the gradients of scores, G and both codebooks
  adamw       an AdamW step over many tensors, states in 32 or in 8 bits

`run` is their plain form in 32-bit torch operations, or the framework's calls where
`own` is true; `exact` is their definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256          # elements that share a scale in the 8-bit states
E4M3_MAX = 448.0
E4M3_MIN = 2.0 ** -9  # the smallest value above zero
TINY = 2.0 ** -100   # a block whose largest value is below this holds zeros
LR, BETA1, BETA2, EPS = 1e-3, 0.9, 0.999, 1e-8
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases --

def listed():
    convs = ",".join(["1024x4096", "2x2x4096"] * 10)  # ten convs' projections and bases at D 4096, group 16
    return [
        # the input rows of one draft block: an anchor and seven mask tokens
        {"name": "embed_block", "op": "embed", "N": 8, "V": 151936, "D": 4096, "table": "bf16", "out": "bf16",
         "scale": 1.0, "masked": 0.875, "pad": 0.0},
        # a training-packed batch of context tokens, scaled, some rows padding
        {"name": "embed_packed", "op": "embed", "N": 16384, "V": 248320, "D": 5120, "table": "bf16", "out": "bf16",
         "scale": 71.554, "masked": 0.0, "pad": 0.02},
        # a smoke-sized step: latency alone
        {"name": "embed_grad_tiny", "op": "embed_grad", "N": 16, "V": 4096, "D": 256, "grad": "f32", "out": "f32",
         "scale": 1.0, "masked": 0.0, "pad": 0.0, "accumulate": False},
        # a ragged micro-batch added to the gradient of earlier ones, rows of an odd length
        {"name": "embed_grad_odd", "op": "embed_grad", "N": 5003, "V": 50021, "D": 251, "grad": "bf16", "out": "f32",
         "scale": 15.8, "masked": 0.0, "pad": 0.1, "accumulate": True},
        # training-packed draft blocks: seven rows of eight are the mask token's
        {"name": "embed_grad_packed", "op": "embed_grad", "N": 16384, "V": 248320, "D": 5120, "grad": "bf16",
         "out": "bf16", "scale": 1.0, "masked": 0.875, "pad": 0.0, "accumulate": False},
        # a smoke-sized selector
        {"name": "selector_tiny", "op": "selector", "P": 16, "K": 4, "r": 32, "V": 4096, "out": "f32",
         "covered": 0.75, "accumulate": False},
        # a micro-batch of 64 blocks of 8 added to the codebooks' gradients
        {"name": "selector_batched", "op": "selector", "P": 512, "K": 16, "r": 256, "V": 248320, "out": "f32",
         "covered": 0.85, "accumulate": True},
        # the training-packed batch: 2048 blocks of 8
        {"name": "selector_packed", "op": "selector", "P": 16384, "K": 16, "r": 256, "V": 151936, "out": "f32",
         "covered": 0.85, "accumulate": False},
        # many candidates and a wide rank, the codebooks' gradients held in bf16
        {"name": "selector_wide", "op": "selector", "P": 4096, "K": 64, "r": 512, "V": 151936, "out": "bf16",
         "covered": 0.9, "accumulate": False},
        # a smoke-sized selector's weights
        {"name": "adamw_tiny", "op": "adamw", "bits": 32, "param": "f32", "grad": "f32", "master": False, "step": 10,
         "shapes": "4096x32,4096x32,32x256,2x2x256"},
        # both codebooks and the hidden projection, bf16 with fp32 master weights, states in 8 bits
        {"name": "adamw_selector_8bit", "op": "adamw", "bits": 8, "param": "bf16", "grad": "f32", "master": True,
         "step": 200, "shapes": "151936x256,151936x256,256x4096"},
        # a drafter's conv weights and many small tensors of odd sizes
        {"name": "adamw_many", "op": "adamw", "bits": 32, "param": "bf16", "grad": "bf16", "master": True, "step": 3,
         "shapes": convs + "," + ",".join("%d" % (1 + 37 * i * i) for i in range(40))},
    ]


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "selector", "adamw"])
    if op in ("embed", "embed_grad"):
        D = log_int(rng, 1, 640) * rng.choice([1, 8])
        N = log_int(rng, 1, min(131072, 16384 * 5120 // D))
        V = log_int(rng, 2, min(248320, 248320 * 5120 // (2 * D)))
        c = {"op": op, "N": N, "V": V, "D": D, "scale": rng.choice([1.0, round(math.sqrt(D), 3), 0.37]),
             "masked": rng.choice([0.0, 0.0, 0.5, 0.875]), "pad": rng.choice([0.0, 0.1])}
        if op == "embed":
            c.update(table=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]))
        else:
            c.update(grad=rng.choice(["bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                     accumulate=rng.random() < 0.5)
        return c
    if op == "selector":
        r = 8 * log_int(rng, 1, 96)
        K = log_int(rng, 1, 128)
        P = log_int(rng, 1, max(1, min(16384, 16384 * 16 * 256 // (K * r))))
        V = log_int(rng, max(K, 16), min(248320, 151936 * 512 // r))
        return {"op": op, "P": P, "K": K, "r": r, "V": V, "out": rng.choice(["bf16", "f32"]),
                "covered": rng.choice([0.0, 0.5, 0.85, 1.0]), "accumulate": rng.random() < 0.5}
    param = rng.choice(["f32", "bf16"])
    n = rng.choice([1, 2, 5, 30, 100])
    shapes = ",".join("%d" % log_int(rng, 1, 20_000_000 // n) if rng.random() < 0.5 else
                      "%dx%d" % (log_int(rng, 1, 20_000_000 // (n * 64)), rng.randint(1, 64)) for _ in range(n))
    return {"op": op, "bits": rng.choice([32, 8]), "param": param, "grad": rng.choice(["f32", "bf16"]),
            "master": param == "bf16" and rng.random() < 0.7, "step": rng.choice([0, 1, 7, 1000]), "shapes": shapes}


def numels(case):
    return [math.prod(int(d) for d in s.split("x")) for s in case["shapes"].split(",")]


# ----------------------------------------------------------------- inputs --

def normal(gen, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0.0, std, generator=gen)
    return x.to(dtype)


def uniform(gen, *shape):
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(0.0, 1.0, generator=gen)


def scatter_rank(rank, V):
    """Ranks by frequency to token ids spread over the vocabulary (a bijection of [0, V))."""
    step = next(q for q in (7919, 104729, 15485863, 1) if math.gcd(q, V) == 1)
    return (rank * step + 11) % V


def tokens(gen, N, V):
    """Token ids whose frequency falls off as 1/rank, as those of text do."""
    rank = torch.exp(uniform(gen, N).double() * math.log(V)).long().clamp_(1, V) - 1
    return scatter_rank(rank, V)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("embed", "embed_grad"):
        N, V, D = case["N"], case["V"], case["D"]
        ids = tokens(gen, N, V)
        ids = torch.where(uniform(gen, N) < case["masked"], torch.full_like(ids, V - 1), ids)
        s["ids"] = torch.where(uniform(gen, N) < case["pad"], torch.full_like(ids, -1), ids).to(torch.int32)
        if op == "embed":
            s["table"] = normal(gen, (V, D), DTYPES[case["table"]], 0.02)
        else:
            s["dout"] = normal(gen, (N, D), DTYPES[case["grad"]], 1e-2)
            s["dtable"] = (normal(gen, (V, D), DTYPES[case["out"]], 1e-2) if case["accumulate"] else
                           torch.empty((V, D), dtype=DTYPES[case["out"]], device="cuda"))
        return s
    if op == "selector":
        P, K, r, V = case["P"], case["K"], case["r"], case["V"]
        # K distinct candidates a row, most of them frequent tokens: one of each of K classes of rank
        j = torch.arange(K, device="cuda", dtype=torch.float64)
        span = V - K + 1
        rank = torch.exp((j + uniform(gen, P, K).double()) / K * math.log(span)).long().clamp_(1, span) - 1
        ids = scatter_rank(rank + torch.arange(K, device="cuda"), V)
        col = (uniform(gen, P) * K).long().clamp_(max=K - 1)
        hit = ids.gather(1, col[:, None])[:, 0]
        s["targets"] = torch.where(uniform(gen, P) < case["covered"], hit, torch.full_like(hit, -1)).to(torch.int32)
        s["topk_ids"] = ids.to(torch.int32)
        s["pred"] = tokens(gen, P, V).to(torch.int32)
        s["topk_vals"] = normal(gen, (P, K), torch.float32, 2.0).sort(dim=1, descending=True).values.contiguous()
        s["G"] = normal(gen, (P, r), torch.float32, 1.3)
        s["A"] = normal(gen, (V, r), torch.bfloat16, 0.3)
        s["Bc"] = normal(gen, (V, r), torch.bfloat16, 0.3)
        s["row_weights"] = uniform(gen, P) / P
        for name in ("dA", "dBc"):
            s[name] = (normal(gen, (V, r), DTYPES[case["out"]], 1e-4) if case["accumulate"] else
                       torch.empty((V, r), dtype=DTYPES[case["out"]], device="cuda"))
        return s
    # adamw: every tensor starts on a block of its own in one flat buffer of each kind
    ns = numels(case)
    starts = np.concatenate([[0], np.cumsum([-(-n // BLOCK) * BLOCK for n in ns])])
    total = int(starts[-1])
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, ns):
        live[int(a):int(a) + n] = True

    def kept(x):
        return torch.where(live, x, torch.zeros_like(x))

    w = kept(normal(gen, total, torch.float32, 0.02))
    s["param"] = w.to(DTYPES[case["param"]])
    s["master"] = w if case["master"] else None
    # gradients a hundred times larger in some blocks than in others; in rare rows exactly zero
    size = torch.exp(uniform(gen, total // BLOCK, 1) * math.log(100.0)) * 1e-4
    g = normal(gen, (total // BLOCK, BLOCK), torch.float32) * size
    g = torch.where(uniform(gen, total // BLOCK, 1) < 0.1, torch.zeros_like(g), g)
    s["grad"] = kept(g.reshape(-1)).to(DTYPES[case["grad"]])
    first = case["step"] == 0
    m = kept((normal(gen, (total // BLOCK, BLOCK), torch.float32) * size * 0.3).reshape(-1)) * (0.0 if first else 1.0)
    v = kept(((normal(gen, (total // BLOCK, BLOCK), torch.float32) * size).square()).reshape(-1)) * (0.0 if first else 1.0)
    if case["bits"] == 8:
        s["m"], s["m_scale"] = to_8bit(m, False)
        s["v"], s["v_scale"] = to_8bit(v.sqrt(), True)
    else:
        s["m"], s["v"] = m, v
    decays = [0.0 if "x" not in shape else 0.01 for shape in case["shapes"].split(",")]
    s["weight_decay"] = decays
    s["keep"] = torch.tensor(np.repeat([1.0 - LR * d for d in decays], [-(-n // BLOCK) for n in ns]),
                             dtype=torch.float32, device="cuda")[:, None]
    s["grad_scale"] = torch.full((1,), 0.73, device="cuda")
    s["step"] = case["step"]

    def parts(x, per=1):
        return [x[int(a) // per:int(a) // per + -(-n // per)] for a, n in zip(starts, ns)]

    s["params"], s["grads"] = parts(s["param"]), parts(s["grad"])
    s["masters"] = parts(s["master"]) if case["master"] else None
    s["state"] = {"exp_avg": parts(s["m"])}
    if case["bits"] == 8:
        s["state"].update(exp_avg_scale=parts(s["m_scale"], BLOCK), exp_avg_rms=parts(s["v"]),
                          exp_avg_rms_scale=parts(s["v_scale"], BLOCK))
    else:
        s["state"].update(exp_avg_sq=parts(s["v"]))
    return s


# ------------------------------------------------------------- plain form --

def to_8bit(x, positive):
    """x as e4m3 values in units of a scale per block; a root above zero never becomes zero."""
    b = x.view(-1, BLOCK)
    top = b.abs().amax(dim=1, keepdim=True)
    held = top >= TINY
    inv = torch.where(held, E4M3_MAX / top, torch.zeros_like(top))
    q = b * inv
    if positive:
        q = torch.where((b > 0) & held, q.clamp(min=E4M3_MIN), q)
    scale = torch.where(held, top / E4M3_MAX, torch.zeros_like(top))
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def from_8bit(q, scale):
    return (q.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def plain_embed(s):
    c = s["case"]
    live = s["ids"] >= 0
    rows = s["table"][s["ids"].clamp(min=0)].float() * c["scale"]
    return torch.where(live[:, None], rows, torch.zeros_like(rows)).to(DTYPES[c["out"]])


def add_rows(ids, rows, V, out, accumulate):
    """out (+)= the sum of the rows of each id, in 32 bits."""
    sums = torch.zeros((V, rows.shape[1]), dtype=torch.float32, device=rows.device)
    sums.index_add_(0, ids, rows)
    out.copy_(out.float() + sums if accumulate else sums)
    return out


def plain_embed_grad(s):
    c = s["case"]
    live = s["ids"] >= 0
    rows = s["dout"].float() * c["scale"]
    rows = torch.where(live[:, None], rows, torch.zeros_like(rows))
    return add_rows(s["ids"].clamp(min=0), rows, c["V"], s["dtable"], c["accumulate"])


def plain_selector(s):
    c = s["case"]
    ids = s["topk_ids"]
    a = s["A"][s["pred"]].float()
    b = s["Bc"][ids].float()                                  # [P, K, r]
    u = a * s["G"]
    scores = s["topk_vals"] + (u[:, None, :] * b).sum(-1)
    is_target = ids == s["targets"][:, None]
    live = is_target.any(1)
    col = torch.where(live, is_target.to(torch.int32).argmax(1), torch.full_like(live, -1, dtype=torch.int64))
    shifted = scores - scores.amax(1, keepdim=True)
    e = shifted.exp()
    total = e.sum(1, keepdim=True)
    loss = total.log()[:, 0] - shifted.gather(1, col.clamp(min=0)[:, None])[:, 0]
    loss = torch.where(live, loss, torch.full_like(loss, float("nan")))
    label = torch.zeros_like(scores).scatter_(1, col.clamp(min=0)[:, None], 1.0)
    ds = torch.where(live[:, None], (e / total - label) * s["row_weights"][:, None], torch.zeros_like(scores))
    t = (ds[:, :, None] * b).sum(1)                           # [P, r]
    dG = a * t
    dA = add_rows(s["pred"], s["G"] * t, c["V"], s["dA"], c["accumulate"])
    dBc = add_rows(ids.reshape(-1), (ds[:, :, None] * u[:, None, :]).reshape(-1, c["r"]), c["V"], s["dBc"],
                   c["accumulate"])
    return {"loss": loss, "label": col.to(torch.int32), "dscores": ds, "dG": dG, "dA": dA, "dBc": dBc}


def plain_adamw(s):
    c = s["case"]
    s["step"] += 1
    w = (s["master"] if c["master"] else s["param"]).float()
    g = s["grad"].float() * s["grad_scale"]
    if c["bits"] == 8:
        m, root = from_8bit(s["m"], s["m_scale"]), from_8bit(s["v"], s["v_scale"])
        v = root * root
    else:
        m, v = s["m"], s["v"]
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * (1.0 - BETA2) * g
    root = v.sqrt()
    denom = root * (1.0 / math.sqrt(1.0 - BETA2 ** s["step"])) + EPS
    w = (w.view(-1, BLOCK) * s["keep"]).view(-1) - m / denom * (LR / (1.0 - BETA1 ** s["step"]))
    if c["master"]:
        s["master"].copy_(w)
    s["param"].copy_(w)
    if c["bits"] == 8:
        for name, x, positive in (("m", m, False), ("v", root, True)):
            q, scale = to_8bit(x, positive)
            s[name].copy_(q)
            s[name + "_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)


def adamw_outputs(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


# -------------------------------------------------------------------- run --

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        if op == "adamw":
            plain_adamw(s)
            return adamw_outputs(s)
        return {"embed": plain_embed, "embed_grad": plain_embed_grad, "selector": plain_selector}[op](s)
    import dflash2_draft_block_gb300 as df2
    if op == "embed":
        return df2.embedding(s["table"], s["ids"], scale=c["scale"], dtype=DTYPES[c["out"]])
    if op == "embed_grad":
        return df2.embedding_grad(s["dout"], s["ids"], c["V"], scale=c["scale"], accumulate=c["accumulate"],
                                  out=s["dtable"])
    if op == "selector":
        loss, label, ds, dG, dA, dBc = df2.selector_loss_grad(
            s["pred"], s["targets"], s["topk_ids"], s["topk_vals"], s["G"], s["A"], s["Bc"],
            row_weights=s["row_weights"], accumulate=c["accumulate"], dA=s["dA"], dBc=s["dBc"])
        return {"loss": loss, "label": label, "dscores": ds, "dG": dG, "dA": dA, "dBc": dBc}
    if "opt" not in s:
        s["opt"] = df2.AdamW(s["params"], s["grads"], lr=LR, betas=(BETA1, BETA2), eps=EPS,
                             weight_decay=s["weight_decay"], state_bits=c["bits"], master_weights=s["masters"],
                             state=s["state"], step=s["step"])
    s["opt"].step(grad_scale=s["grad_scale"])
    return adamw_outputs(s)


# ------------------------------------------------------------------- work --

def distinct(N, V, masked=0.0):
    """Expected number of different ids among N drawn by tokens()."""
    n = N * (1.0 - masked)
    rank = np.arange(1, V + 1, dtype=np.float64)
    p = np.log((rank + 1) / rank) / math.log(V)
    return float(np.sum(-np.expm1(-n * np.minimum(p, 1.0)))) + (1.0 if masked else 0.0)


def work(case):
    op = case["op"]
    if op in ("embed", "embed_grad"):
        N, V, D = case["N"], case["V"], case["D"]
        rows = min(N, distinct(N * (1.0 - case["pad"]), V, case["masked"]))
        if op == "embed":
            return {"bytes": 4 * N + rows * D * SIZES[case["table"]] + N * D * SIZES[case["out"]], "flops": N * D}
        o = SIZES[case["out"]]
        table = 2 * rows * D * o if case["accumulate"] else V * D * o
        return {"bytes": 4 * N + N * (1.0 - case["pad"]) * D * SIZES[case["grad"]] + table, "flops": 2 * N * D}
    if op == "selector":
        P, K, r, V = case["P"], case["K"], case["r"], case["V"]
        o = SIZES[case["out"]]
        span = V - K + 1
        live = P * case["covered"]
        # expected different candidates: class j holds ranks span^(j/K) .. span^((j+1)/K), drawn once a row
        cand = 0.0
        for j in range(K):
            lo, hi = span ** (j / K), span ** ((j + 1) / K)
            k = np.arange(math.floor(lo), math.ceil(hi) + 1, dtype=np.float64)
            p = np.maximum(0.0, np.log(np.minimum(k + 1, hi) / np.maximum(k, lo))) / math.log(max(span, 2)) * K
            cand += float(np.sum(1.0 - (1.0 - np.minimum(p, 1.0)) ** live))
        cand = min(cand, V, live * K)
        preds = min(distinct(live, V), live)
        grads = 2 * (preds + cand) * r * o if case["accumulate"] else 2 * V * r * o
        # ids, values and dscores a candidate; pred, target, weight, loss and label a row; G in, dG out
        return {"bytes": 12 * P * K + 20 * P + (live + P) * r * 4 + (preds + cand) * r * 2 + grads,
                "flops": live * K * r * 6 + live * r * 3}
    n = sum(numels(case))
    per = 2 * (8 if case["bits"] == 32 else 2 + 8 / BLOCK) + SIZES[case["grad"]]
    per += 8 + SIZES[case["param"]] if case["master"] else 2 * SIZES[case["param"]]
    return {"bytes": n * per, "flops": 14 * n}


# ------------------------------------------------------------------ exact --

def exact_sums(index, contributions, V):
    """[V, D] in 64 bits: the contributions of each id, as differences of their running sums in the order of a sort by id."""
    out = torch.zeros((V, contributions.shape[1]), dtype=torch.float64, device=contributions.device)
    order = torch.argsort(index, stable=True)
    names, counts = torch.unique_consecutive(index[order], return_counts=True)
    ends = counts.cumsum(0)
    running = torch.nn.functional.pad(contributions[order].cumsum(0), (0, 0, 1, 0))
    out[names] = running[ends] - running[ends - counts]
    return out


def e4m3(x):
    """x >= 0 in 64 bits to the nearest e4m3 value, ties to even."""
    exp = torch.frexp(x.clamp(min=E4M3_MIN))[1].double()
    ulp = torch.exp2((exp - 1).clamp(min=-6) - 3)
    return (torch.round(x / ulp) * ulp).clamp(max=E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        ids = s["ids"].long()
        out = torch.zeros((case["N"], case["D"]), dtype=torch.float64, device="cuda")
        out[ids >= 0] = s["table"].index_select(0, ids[ids >= 0]).double() * case["scale"]
        return out
    if op == "embed_grad":
        ids = s["ids"].long()
        got = exact_sums(ids[ids >= 0], s["dout"][ids >= 0].double() * case["scale"], case["V"])
        return got + s["dtable"].double() if case["accumulate"] else got
    if op == "selector":
        P, K, r, V = case["P"], case["K"], case["r"], case["V"]
        found = s["topk_ids"] == s["targets"][:, None]
        live = found.any(1).nonzero()[:, 0]
        G, a = s["G"].double()[live], s["A"][s["pred"].long()].double()[live]
        b = s["Bc"][s["topk_ids"].long()[live]].double()
        score = s["topk_vals"].double()[live] + torch.bmm(b, (a * G)[:, :, None])[:, :, 0]
        hit = found[live].double()
        loss = torch.full((P,), float("nan"), dtype=torch.float64, device="cuda")
        loss[live] = torch.logsumexp(score, 1) - (score * hit).sum(1)
        d = (torch.softmax(score, 1) - hit) * s["row_weights"].double()[live][:, None]
        t = torch.bmm(d[:, None, :], b)[:, 0]
        ds = torch.zeros((P, K), dtype=torch.float64, device="cuda")
        ds[live] = d
        dG = torch.zeros((P, r), dtype=torch.float64, device="cuda")
        dG[live] = a * t
        dA = exact_sums(s["pred"].long()[live], G * t, V)
        del b
        dBc = torch.zeros((V, r), dtype=torch.float64, device="cuda")
        for k in range(K):
            dBc += exact_sums(s["topk_ids"].long()[live, k], d[:, k, None] * (a * G), V)
        if case["accumulate"]:
            dA, dBc = dA + s["dA"].double(), dBc + s["dBc"].double()
        return {"loss": loss, "label": None, "dscores": ds, "dG": dG, "dA": dA, "dBc": dBc}
    w = (s["master"] if case["master"] else s["param"]).double()
    m = s["m"].float().double().view(-1, BLOCK)
    v = s["v"].float().double().view(-1, BLOCK)
    if case["bits"] == 8:
        m = m * s["m_scale"].double()[:, None]
        v = (v * s["v_scale"].double()[:, None]) ** 2
    t = case["step"] + 1
    g = (s["grad"].double() * s["grad_scale"].double()).view(-1, BLOCK)
    m = BETA1 * m + (1.0 - BETA1) * g
    v = BETA2 * v + (1.0 - BETA2) * g ** 2
    update = (m / (1.0 - BETA1 ** t)) / ((v / (1.0 - BETA2 ** t)).sqrt() + EPS)
    decay = torch.tensor(np.repeat(s["weight_decay"], [-(-n // BLOCK) for n in numels(case)]), device="cuda")
    w = w.view(-1, BLOCK)
    w = (w - LR * (update + decay[:, None] * w)).view(-1)
    out = {"param": w, "m": m.view(-1), "v": v.view(-1)}
    if case["bits"] == 8:
        for name, x in (("m", m), ("v", v.sqrt())):
            top = x.abs().amax(1, keepdim=True)
            unit = torch.where(top >= TINY, top / E4M3_MAX, torch.zeros_like(top))
            y = torch.where(unit > 0, x / unit, torch.zeros_like(x))
            q = e4m3(y.abs())
            if name == "v":
                q = torch.where((y > 0) & (q == 0), torch.full_like(q, E4M3_MIN), q)
            out[name], out[name + "_scale"] = (torch.sign(y) * q).view(-1), unit.view(-1)
    if case["master"]:
        out["master"] = w
    return out
