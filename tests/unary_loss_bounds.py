"""How far the unary loss may be from its definition, with sums in pieces as the kernels make them.

The tensor core adds 16 products a step and cuts a partial sum below its last bit: at most 2^-23 of the
sum of its terms' sizes, S.  A sum of n products in pieces of c is off by c / 16 such cuts, by a
rounding to nearest (2^-24 of S) for each piece added, and by a few more: steps(n, c) 2^-23 S.
Logits are summed 1,024 products at a time, dh and dW 4,096; a tile of dh may also be cut into up to
64 parts, each added once.

A logit's map rounds a few times (2^-21 of it) and steepens by m at most.  exp's argument is rounded
(2^-22 of the difference from its tile's and the row's largest), sums of exponentials are trees of a few
dozen roundings (2^-18).  The softcap's slope m / cosh^2 y has a relative error of twice y's, |y| 2^-20
from exp and 2^-19 from a few roundings more.  A factor g is exp(x - lse) times the slope, rounded to
fp16 (2^-11, and 2^-40 of the row's largest exp(x - lse) m), with the row's weight (2^-15 for that and
a few products) and to bf16 (2^-8)."""
import torch


def steps(n, piece):
    return (min(n, piece) + 15) // 16 + n / piece / 2 + 4


def definition(h, W, targets, weights=None, mul=1.0, cap=0.0):
    """(loss, lse, dh, dW) in 64 bits and a dict of bounds, on h's device."""
    P, D = h.shape
    V = W.shape[0]
    live = (targets >= 0) & (targets < V)
    zero = torch.zeros((), dtype=torch.float64, device=h.device)
    h = torch.where(live[:, None], h.double(), zero)
    W = W.double()
    t = torch.where(live, targets, torch.zeros_like(targets)).long()[:, None]
    w = torch.where(live, (torch.ones(P, device=h.device) if weights is None else weights).double(), zero)[:, None]
    u = h @ W.T
    y = mul * u / cap if cap else zero
    x = cap * torch.tanh(y) if cap else mul * u
    slope = mul / torch.cosh(y) ** 2 if cap else torch.full_like(u, mul)
    du = steps(D, 1024) * 2.0 ** -23 * (h.abs() @ W.abs().T)
    # (a logit of the target's tile is mapped as any other: the errors of a row's logits are alike)
    dx = mul * du + 2.0 ** -21 * x.abs()
    rel_slope = 2 * mul * du / cap + 2.0 ** -20 * y.abs() + 2.0 ** -19 if cap else zero
    worst, top = dx.amax(1, keepdim=True), x.amax(1, keepdim=True)
    lse = torch.logsumexp(x, 1, keepdim=True)
    drop = 2.0 ** -21 * (top - x)
    p = torch.exp(x - lse)
    xt = x.gather(1, t)
    others = torch.logsumexp(x.scatter(1, t, -float("inf")), 1, keepdim=True) if V > 1 else torch.full_like(xt, -float("inf"))
    loss = torch.logaddexp(torch.zeros_like(xt), others - xt)
    p_others = torch.exp(others - lse).clamp(max=1.0)
    dlse = worst + (p * drop).sum(1, keepdim=True) + 2.0 ** -18 + 2.0 ** -22 * (lse.abs() + top.abs())
    dloss = p_others * (2 * worst + (p * drop).sum(1, keepdim=True) + 2.0 ** -18) + 2.0 ** -22 * (loss + (top - xt)) + 1e-38
    g = p.scatter(1, t, -p_others)
    dg = g.abs() * slope * (dx + worst + drop + 2.0 ** -17 + rel_slope + 2.0 ** -11 + 2.0 ** -15 + 2.0 ** -8)
    dg = (dg + mul * 2.0 ** -40 * torch.exp(top - lse)) * w.abs() + torch.where(live, 1e-38, 0.0)[:, None]
    g = g * slope * w
    dh, dW = g @ W, g.T @ h
    ddh = (dg + (steps(V, 4096) + 32) * 2.0 ** -23 * g.abs()) @ W.abs()
    ddW = (dg + steps(P, 4096) * 2.0 ** -23 * g.abs()).T @ h.abs()
    nan = torch.full_like(loss, float("nan"))
    return (torch.where(live[:, None], loss, nan)[:, 0], torch.where(live[:, None], lse, nan)[:, 0], dh, dW), \
        dict(loss=dloss[:, 0], lse=dlse[:, 0], dh=ddh, dW=ddW)


def check(name, got, want, room):
    """got within room of want and half a step of its own type; NaN in the same places."""
    got64 = got.double()
    assert torch.equal(got64.isnan(), want.isnan()), f"{name}: NaN in other places"
    half = torch.finfo(got.dtype).eps / 2
    room = room + half * (want.abs() + room) + 1e-38
    off = ((got64 - want).abs() / room)[~want.isnan()]
    assert not off.numel() or float(off.max()) <= 1.0, f"{name}: off by {float(off.max()):.3g} of what roundings allow"
