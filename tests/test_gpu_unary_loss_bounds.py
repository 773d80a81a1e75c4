"""The unary loss against its definition in 64 bits, within what sums in pieces allow (unary_loss_bounds):
sums of one sign that would show a piece that is too long, sums that any part left out or taken twice
would change, and the far ends of the stated range."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from unary_loss_bounds import check, definition, steps  # noqa: E402

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


def inputs(seed, P, V, D, spread=2.5, raised=12.0, masked=0.2):
    """Logits of deviation `spread`, targets raised by up to `raised`, a share without a target."""
    g = torch.Generator().manual_seed(seed)
    W = (torch.randn(V, D, generator=g) * (spread / D ** 0.5)).to(BF)
    t = torch.randint(0, V, (P,), generator=g)
    up = torch.rand(P, 1, generator=g) * raised / spread ** 2
    h = (torch.randn(P, D, generator=g) + up * W[t].float()).to(BF)
    t = torch.where(torch.rand(P, generator=g) < masked, torch.full_like(t, -1), t).to(I32)
    return h.cuda(), W.cuda(), t.cuda(), (torch.rand(P, generator=g) * 2).cuda()


@pytest.mark.parametrize("mul, cap", [(1.0, 0.0), (0.8, 30.0), (2.0, 3.0)])
@pytest.mark.parametrize("P, V, D", [(1, 1, 8), (8, 1000, 72), (33, 129, 4096), (130, 777, 1032), (300, 2050, 2504),
                                     (7, 40001, 264), (70, 20000, 520), (500, 9001, 136), (5000, 700, 200), (9100, 513, 1160)])
def test_sizes(df2, P, V, D, mul, cap):
    h, W, t, w = inputs(P + V, P, V, D)
    want, room = definition(h, W, t, w, mul, cap)
    for dtype in (BF, F32):
        got = df2.unary_loss_grad(h, W, t, row_weights=w, output_multiplier=mul, final_logit_softcapping=cap, dW=True,
                                  dtype=dtype)
        for n, a, b in zip(("loss", "lse", "dh", "dW"), got, want):
            check(n, a, b, room[n])


@pytest.mark.parametrize("D", [1024, 4096, 1 << 16, (1 << 20) - 8])
def test_a_logit_is_summed_in_pieces(df2, D):
    """One column: the log-sum-exp is its logit, here a sum of one sign.  (2^16 terms of one sign in one
    piece, as dW's were, came out 3.4e-4 too small; pieces of 1,024 allow 1.2e-5.)"""
    g = torch.Generator().manual_seed(D)
    h, W = ((torch.rand(n, D, generator=g) + 0.5).to(BF).cuda() for n in (40, 1))
    t = torch.zeros(40, dtype=I32, device="cuda")
    loss, lse = df2.unary_ce(h, W, t)
    want = (h.double() @ W.double().T)[:, 0]
    assert not bool(loss.any())
    off = ((lse.double() - want) / want).abs().max()
    assert float(off) <= steps(D, 1024) * 2.0 ** -23 + 2.0 ** -23, float(off)


@pytest.mark.parametrize("P, V, D", [(1, 1 << 12, 8), (8, 1 << 15, 1032), (40, 1 << 17, 256), (300, 1 << 16, 520),
                                     (600, 1 << 12, 4104), (1500, 1 << 14, 2568), (8, 1 << 20, 64), (3, 1 << 22, 8)])
def test_every_part_of_dh_counts_once(df2, P, V, D):
    """Equal columns: a factor is w / V, the target's -w (1 - 1 / V) rounded to -w, and W's row is v's
    place, or one: sums that are exact (no more than 24 bits from 1 / V to the largest; past 2^17 columns
    the targets are where that place is 0), so a step left out or summed twice shows whole."""
    g = torch.Generator().manual_seed(V)
    h = torch.zeros(P, D, dtype=BF, device="cuda")
    W = torch.ones(V, D, dtype=BF, device="cuda")
    W[:, 1] = (torch.arange(V) * 64 // V).to(BF).cuda()  # which 64th of the columns
    t = torch.randint(0, V if V <= 1 << 17 else V // 64, (P,), generator=g).to(I32).cuda()
    dh = df2.unary_loss_grad(h, W, t, dtype=F32)[2].double()
    want = W.double().sum(0) / V - (1 + 1 / V) * W[t.long()].double()
    assert torch.equal(dh, want)


def test_most_rows(df2):
    """2^20 rows, of which 7 of 10 have a target: each block puts many in order, and dW sums them all."""
    P, V, D = 1 << 20, 9, 8
    h, W, t, w = inputs(51, P, V, D, masked=0.3)
    want, room = definition(h, W, t, w)
    got = df2.unary_loss_grad(h, W, t, row_weights=w, dW=True, dtype=F32)
    for n, a, b in zip(("loss", "lse", "dh", "dW"), got, want):
        check(n, a, b, room[n])
    with pytest.raises(df2.DFlash2Error):
        df2.unary_ce(torch.zeros(P + 1, D, dtype=BF, device="cuda"), W, torch.zeros(P + 1, dtype=I32, device="cuda"))


@pytest.mark.parametrize("masked", [0.0, 0.6])
def test_capped_pieces(df2, masked):
    """2^22 columns under a softcap: 700 rows go in two pieces, each with its targets' slopes."""
    P, V, D = 700, 1 << 22, 8
    h, W, t, w = inputs(52, P, V, D, masked=masked)
    got = df2.unary_loss_grad(h, W, t, row_weights=w, final_logit_softcapping=4.0, dW=True, dtype=F32)
    dW = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    room_dW = torch.zeros_like(dW)
    for some in torch.arange(P, device="cuda").split(50):
        want, room = definition(h[some], W, t[some], w[some], 1.0, 4.0)
        for n, i in (("loss", 0), ("lse", 1), ("dh", 2)):
            check(n, got[i][some], want[i], room[n])
        dW += want[3]
        room_dW += room["dW"] * (1 + 2.0 ** -9)  # (512 rows' steps, beside 2^-8 of each factor)
    check("dW", got[3], dW, room_dW + 2.0 ** -22 * dW.abs())


def test_what_is_not_finite_in_the_head(df2):
    """A NaN in one of W's rows is in every row's sum; a row that makes its logits -infinity is as if it
    were not there."""
    h, W, t, w = inputs(53, 90, 600, 64, masked=0.2)
    live = t >= 0
    bad = W.clone()
    bad[37, 5] = float("nan")
    loss, lse, dh, dW = df2.unary_loss_grad(h, bad, t, dW=True)
    assert bool(loss.isnan().all()) and bool(lse.isnan().all()) and bool(dh[live].isnan().all()) and not bool(dh[~live].any())
    gone = torch.tensor([0, 63, 64, 127, 300, 599], device="cuda")
    some = torch.ones(600, dtype=torch.bool, device="cuda")
    some[gone] = False
    t = torch.where(live & some[t.clamp(min=0).long()], t, torch.full_like(t, -1))
    far_h, far_W = torch.cat([h, torch.ones_like(h[:, :8])], 1), torch.cat([W, torch.zeros_like(W[:, :8])], 1)
    for low in (-float("inf"), -3e38):
        far_W[gone, 64] = low
        far_h[:, 64] = 1.0 if low == -float("inf") else 2.0 ** 10
        loss, lse, dh, dW = df2.unary_loss_grad(far_h, far_W, t, row_weights=w, dW=True, dtype=F32)
        number = torch.cumsum(some.long(), 0) - 1
        less = torch.where(t >= 0, number[t.clamp(min=0).long()], torch.full_like(t, -1).long()).to(I32)
        want, room = definition(h, W[some], less, w)
        check("loss", loss, want[0], room["loss"])
        check("lse", lse, want[1], room["lse"])
        check("dh", dh[:, :64], want[2], room["dh"])
        check("dW", dW[some][:, :64], want[3], room["dW"])
        assert not bool(dW[gone][:, :64].any())
