"""The unary loss and its gradients from their definition in 64 bits, with how far fp32 sums
and the bf16 factors of the products may take a result from it.

A logit is a sum of exact products in D / 16 steps of the tensor core, each cut below the last
bit of a partial sum (2^-23 of it, and it is at most S = sum |h W|), added up in fp32:
du = (D / 16 + 4) 2^-23 S.  The map multiplies by m (slope at most m) and rounds a few times:
dx = m du + 2^-21 |x|.  exp turns dx, and the 2^-22 of its argument's product, into relative
errors; a log-sum-exp is off by no more than its worst term, plus the rounding of sums of V
terms in a tree of 64 columns a thread and of results of size |lse| and |x_t|.
A factor g is exp(x - lse) to those relative errors, rounded to fp16 (2^-11 of it, and in units of
2^-39 of the largest of its 64 columns, which is at most the row's) and then to bf16 (2^-8);
products of them are summed in n / 16 steps like the logits.
"""
import torch


def reference(h, W, targets, weights=None, mul=1.0, cap=0.0, dW0=None):
    """(loss, lse, dh, dW) and a dict of bounds, in 64 bits, on h's device."""
    P, D = h.shape
    V = W.shape[0]
    live = (targets >= 0) & (targets < V)
    h = torch.where(live[:, None], h.double(), torch.zeros((), dtype=torch.float64, device=h.device))
    W = W.double()
    t = torch.where(live, targets, torch.zeros_like(targets)).long()
    w = (torch.ones(P, device=h.device) if weights is None else weights).double()
    w = torch.where(live, w, torch.zeros_like(w))
    u = h @ W.T
    du = (D / 16 + 4) * 2.0 ** -23 * (h.abs() @ W.abs().T)
    x = cap * torch.tanh(mul * u / cap) if cap else mul * u
    slope = mul * (1.0 - (x / cap) ** 2) if cap else torch.full_like(x, mul)
    dx = mul * du + 2.0 ** -21 * x.abs()
    lse = torch.logsumexp(x, 1)
    xt = x.gather(1, t[:, None])[:, 0]
    others = torch.logsumexp(x.scatter(1, t[:, None], -float("inf")), 1) if V > 1 else torch.full_like(xt, -float("inf"))
    loss = torch.logaddexp(torch.zeros_like(xt), others - xt)
    top = x.amax(1)
    drop = 2.0 ** -22 * (top[:, None] - x).abs()                # of the exponent's product
    rel = dx + dx.amax(1, keepdim=True) + drop + 2.0 ** -18      # of exp(x - lse): sums of 2^7 + 2^5 roundings
    dlse = dx.amax(1) + (torch.softmax(x, 1) * drop).sum(1) + 2.0 ** -18 + 2.0 ** -22 * (lse.abs() + top.abs())
    p_others = torch.exp(others - lse)
    # the loss moves by the others' share of the logits' difference
    dloss = p_others.clamp(max=1.0) * (2 * dx.amax(1) + 2.0 ** -18) + 2.0 ** -22 * (loss + (top - xt)) + 1e-38
    g = torch.exp(x - lse[:, None])
    g.scatter_(1, t[:, None], -p_others[:, None])
    # the slope 1 - (x / c)^2 from a rounded x
    dslope = 2 * mul * x.abs() * dx / cap ** 2 + 2.0 ** -21 * mul if cap else torch.zeros_like(x)
    dg = g.abs() * (slope * (rel + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15) + dslope) + mul * 2.0 ** -40 * torch.exp(top - lse)[:, None]
    g, dg = g * slope * w[:, None], dg * w.abs()[:, None] + 1e-38
    dh, dW = g @ W, g.T @ h
    ddh = (dg + (V / 16 + 4) * 2.0 ** -23 * g.abs()) @ W.abs()
    ddW = (dg + (P / 16 + 4) * 2.0 ** -23 * g.abs()).T @ h.abs()
    if dW0 is not None:
        dW = dW + dW0.double()
    nan = torch.full_like(loss, float("nan"))
    return (torch.where(live, loss, nan), torch.where(live, lse, nan), dh, dW), \
        dict(loss=dloss, lse=dlse, dh=ddh, dW=ddW)


HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(name, got, want, room):
    """got within room of want, and half a step of its own type; NaN in the same places."""
    got64 = got.double()
    assert torch.equal(got64.isnan(), want.isnan()), f"{name}: NaN in other places"
    ok = ~want.isnan()
    off = (got64 - want)[ok].abs()
    room = room.expand_as(want)[ok]
    room = room * (1 + HALF_STEP[got.dtype]) + 2 * HALF_STEP[got.dtype] * want[ok].abs() + 1e-38
    assert bool((off <= room).all()), f"{name}: off by {float((off / room).max()):.3g} of what roundings allow"
    return float((off / room).max()) if off.numel() else 0.0
