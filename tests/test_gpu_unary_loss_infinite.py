"""Logits of infinite size: under a softcap they are -c and c like any other that saturates it, and
without one a logit of -infinity has no share.

Every logit here is one product, exact in fp32, or overflows, so its only error is the map's: 2^-20 of
the cap.  A log-sum-exp is off by that and 2^-17 (exponentials, and sums of a few hundred terms), a
loss by twice as much.  A factor g is off by those as relative errors, by its rounding to fp16 and
bf16, by 2^-40 of the row's largest, and by its slope's error, 2^-19 of the multiplier at most."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FAR = 2.0 ** 80  # its square is past fp32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


def inputs(V, kinds, far=FAR):
    """Rows whose logits are W[:, 1] (h = far, 1) or plain (h = 0, 1); kinds[v] is -1, 0 or 1: the sign
    of the infinity that column v has in the far rows.  Targets: every fifth column."""
    g = torch.Generator().manual_seed(V)
    W = torch.zeros(V, 8)
    W[:, 0] = kinds.float() * FAR
    W[:, 1] = torch.randn(V, generator=g) * 3
    targets = torch.arange(0, V, 5).repeat(2)
    h = torch.zeros(len(targets), 8)
    h[:, 1] = 1.0
    h[: len(targets) // 2, 0] = far
    return h.to(BF).cuda(), W.to(BF).cuda(), targets.to(I32).cuda()


def check(df2, h, W, t, kinds, mul, cap):
    far = h[:, 0] != 0
    x = mul * W[:, 1].double().expand(len(h), -1)
    infinite = far[:, None] & (kinds != 0).cuda()
    u = torch.where(infinite, kinds.cuda() * float("inf"), x)
    if cap:
        y = torch.tanh(u / cap)
        u, slope = cap * y, mul * (1.0 - y * y)
    else:
        slope = torch.full_like(u, mul)
    lse = torch.logsumexp(u, 1)
    xt = u.gather(1, t.long()[:, None])[:, 0]
    g = torch.exp(u - lse[:, None])
    g.scatter_add_(1, t.long()[:, None], -torch.ones_like(lse)[:, None])
    eps = 2.0 ** -20 * (cap or float(x.abs().max())) + 2.0 ** -17
    dg = (g * slope).abs() * (2 * eps + 2.0 ** -8 + 2.0 ** -11) + mul * 2.0 ** -40
    if cap:
        dg += mul * 2.0 ** -19 * g.abs()
    g = g * slope
    for dtype in (BF, F32):
        loss, l, dh, dW = df2.unary_loss_grad(h, W, t, output_multiplier=mul, final_logit_softcapping=cap, dW=True,
                                              dtype=dtype)
        assert torch.equal(torch.stack(df2.unary_ce(h, W, t, output_multiplier=mul, final_logit_softcapping=cap)).nan_to_num(
            -1.0, 1e30), torch.stack((loss, l)).nan_to_num(-1.0, 1e30))
        finite = xt.isfinite()
        assert bool(((l - lse).abs() <= eps).all())
        assert bool(((loss - (lse - xt)).abs() <= 2 * eps)[finite].all()) and bool((loss[~finite] == float("inf")).all())
        half = torch.finfo(dtype).eps / 2
        # (without the far column)
        want, room = g @ W[:, 1:].double(), (dg + 2.0 ** -18 * g.abs()) @ W[:, 1:].double().abs()
        assert bool(((dh[:, 1:] - want).abs() <= room * (1 + half) + half * want.abs() + 1e-38).all())
        want, room = g.T @ h[:, 1:].double(), (dg + 2.0 ** -18 * g.abs()).T @ h[:, 1:].double().abs()
        assert bool(((dW[:, 1:] - want).abs() <= room * (1 + half) + half * want.abs() + 1e-38).all())


@pytest.mark.parametrize("far", [FAR, -FAR, float("inf")])
@pytest.mark.parametrize("V", [1, 5, 64, 65, 200, 256, 777])
@pytest.mark.parametrize("mul, cap", [(1.0, 5.0), (0.5, 30.0)])
def test_capped(df2, V, mul, cap, far):
    """All of them infinite; one sign in some places; whole tiles of 64 columns; both signs."""
    g = torch.Generator().manual_seed(7)
    sign = 1 if far > 0 else -1
    every = [torch.full((V,), -sign), torch.full((V,), sign), torch.where(torch.rand(V, generator=g) < 0.3, -sign, 0),
             torch.where(torch.arange(V) // 64 % 2 == 1, -sign, 0), torch.randint(-1, 2, (V,), generator=g)]
    for kinds in every:
        if far == float("inf") and bool((kinds == 0).any()):
            continue  # infinity times nothing
        h, W, t = inputs(V, kinds, far)
        check(df2, h, W, t, sign * kinds, mul, cap)


def test_all_capped_from_below(df2):
    """Every logit -infinity: all equal, so the loss is the logarithm of their number."""
    V = 300
    h, W, t = inputs(V, torch.full((V,), -1))
    loss, lse = df2.unary_ce(h, W, t, final_logit_softcapping=8.0)
    far = h[:, 0] != 0
    assert bool(((loss[far] - 5.703782474656201).abs() < 2.0 ** -16).all())
    assert bool(((lse[far] - 5.703782474656201 + 8.0).abs() < 2.0 ** -16).all())


@pytest.mark.parametrize("V", [5, 65, 200, 777])
@pytest.mark.parametrize("mul", [1.0, 0.5])
def test_uncapped(df2, V, mul):
    """-infinity in some columns, and in whole tiles: they have no share; as a target, an infinite loss."""
    g = torch.Generator().manual_seed(8)
    for kinds in (torch.where(torch.rand(V, generator=g) < 0.3, -1, 0), torch.where(torch.arange(V) // 64 % 2 == 1, -1, 0)):
        kinds[V - 1] = 0
        h, W, t = inputs(V, kinds)
        check(df2, h, W, t, kinds, mul, 0.0)
