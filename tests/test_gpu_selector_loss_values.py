"""The selector's loss where fp32 could lose it: scores far from zero, rows of nothing but
the lowest fp32, NaN.

With G = 0 the scores are topk_vals themselves, so the loss in 64 bits of the same fp32
scores is what a call should give.  Tolerance, with U = 2^-24 and d_j = s_j - max s: each
difference is rounded once (U |d_j|, which moves exp by as much of itself), expf is within
2 ulp (4 U), a sum of K positive terms within K U, logf within 1 ulp (2 U) of its value, and
max s - s_label and the last sum are rounded once each."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, F64 = torch.float32, torch.float64
LOW = torch.finfo(F32).min


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    m.lib()
    return m


def case(seed, P, K, r, V):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.rand(P, V, generator=gen, device="cuda").topk(K, dim=1).indices.to(torch.int32).contiguous()
    col = torch.randint(0, K, (P, 1), generator=gen, device="cuda")
    return dict(pred=torch.randint(0, V, (P,), generator=gen, device="cuda", dtype=torch.int32),
                targets=ids.gather(1, col)[:, 0].contiguous(), topk_ids=ids,
                topk_vals=torch.randn(P, K, generator=gen, device="cuda") * 2,
                G=torch.randn(P, r, generator=gen, device="cuda"),
                A=torch.randn(V, r, generator=gen, device="cuda").to(torch.bfloat16),
                Bc=torch.randn(V, r, generator=gen, device="cuda").to(torch.bfloat16)), col[:, 0]


def scores(offset, P, K, gen):
    s = torch.randn(P, K, generator=gen, device="cuda") * 2
    return torch.full_like(s, LOW) if offset == "lowest" else s + offset


def near_loss(loss, s, col):
    s = s.to(F64)
    K = s.shape[1]
    top = s.amax(1, keepdim=True)
    d = s - top
    e = d.exp()
    total = e.sum(1)
    gap = -d.gather(1, col[:, None])[:, 0]
    want = total.log() + gap
    tol = U * (K + 4 + (e * d.abs()).sum(1) / total + 2 * total.log() + gap + want)
    off = (loss.to(F64) - want).abs() - tol
    assert torch.all(off <= 0), f"{float(off.max())} over, of a loss of {float(want[off.argmax()])}"


OFFSETS = [0.0, 1000.0, -1000.0, 3e4, "lowest"]


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("P, K, r", [(40, 16, 64), (30, 2, 256), (9, 100, 520), (700, 16, 256)])
def test_the_loss_of_scores_far_from_zero(df2, offset, P, K, r):
    c, col = case(P + K, P, K, r, 300)
    gen = torch.Generator(device="cuda").manual_seed(3)
    c["topk_vals"] = scores(offset, P, K, gen)
    c["G"].zero_()
    loss, label, ds, *_ = df2.selector_loss_grad(**c)
    assert torch.equal(label.long(), col)
    near_loss(loss, c["topk_vals"], col)
    if offset == "lowest":
        want = torch.full((P, K), 1.0 / K, device="cuda").scatter_add_(1, col[:, None], torch.full((P, 1), -1.0, device="cuda"))
        assert torch.all((ds - want).abs() <= 8 * U)


@pytest.mark.parametrize("offset", OFFSETS)
@pytest.mark.parametrize("P, K", [(40, 16), (30, 2), (9, 100), (3, 1000)])
def test_the_forward_call_of_scores_far_from_zero(df2, offset, P, K):
    c, col = case(P + K, P, K, 8, 1100)
    s = scores(offset, P, K, torch.Generator(device="cuda").manual_seed(3))
    loss, label = df2.selector_ce(s, c["topk_ids"], c["targets"], 1100)
    assert torch.equal(label.long(), col)
    near_loss(loss, s, col)


@pytest.mark.parametrize("P, K, r", [(20, 16, 64), (200, 16, 256), (20, 70, 520)])
def test_nan_scores_are_no_missing_target(df2, P, K, r):
    """A covered row whose scores hold a NaN, all of them or one, keeps its label, and its
    loss and gradients are NaN; the other rows are what they are without it."""
    V = 4000
    c, col = case(P, P, K, r, V)
    c["pred"] = torch.arange(P, device="cuda", dtype=torch.int32) * 3
    clean = df2.selector_loss_grad(**c)
    c["G"][0, r - 1] = float("nan")                  # one value reaches every score
    c["topk_vals"][1] = float("nan")
    c["topk_vals"][2, K // 2] = float("nan")
    c["topk_vals"][3] = float("-inf")
    c["topk_vals"][3, K - 1] = float("nan")
    c["A"][12, 0] = float("nan")                     # row 4's predecessor
    c["topk_vals"][5] = float("-inf")                # nothing to learn: dropped, as before
    loss, label, ds, dG, dA, dBc = df2.selector_loss_grad(**c)
    nan = torch.arange(P, device="cuda") < 5
    keep = torch.arange(P, device="cuda") > 5
    assert torch.equal(label[nan].long(), col[nan]) and int(label[5]) == -1
    assert torch.all(loss[:6].isnan()) and torch.all(ds[nan].isnan()) and torch.all(dG[nan].isnan())
    assert torch.all(ds[5] == 0) and torch.all(dG[5] == 0)
    for got, was in zip((loss, label, ds, dG), clean):
        assert torch.equal(got[keep], was[keep])
    at = torch.zeros(V, dtype=torch.bool, device="cuda")
    at[c["pred"][nan].long()] = True
    assert torch.all(dA[at].isnan()) and torch.all(dA[~at].isfinite())
    at = torch.zeros(V, dtype=torch.bool, device="cuda")
    at[c["topk_ids"][nan].long().view(-1)] = True
    assert torch.all(dBc[at].isnan()) and torch.all(dBc[~at].isfinite())
