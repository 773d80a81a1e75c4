"""The unary loss's long sums, where every term has one sign and every factor is exact, so that nothing
but the sums themselves can be off.

A step of 16 products on the tensor core cuts a sum off below its last bit: at most 2^-23 of it.
Sums in pieces of n steps, the pieces added in fp32 rounded to nearest (2^-24), are off by no more than
n 2^-23 and 2^-24 for each piece, a sum in one piece by n / 4 of its last bits, all downwards."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def df2():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dflash2_draft_block_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P, V, D", [(5000, 256, 72), (1 << 16, 512, 64), (1 << 18, 256, 64), ((1 << 20) - 17, 64, 8),
                                     (9000, 1 << 18, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_dw_of_many_rows(df2, P, V, D, dtype, accumulate):
    """W = 0: every probability is 1 / V, and with weights of 8 bits every factor but the target's is
    exact.  4,096 rows (256 steps) to a piece."""
    g = torch.Generator().manual_seed(P)
    h = (torch.rand(P, D, generator=g) + 0.5).to(BF).cuda()
    w = (torch.rand(P, generator=g) + 0.5).to(BF).float().cuda()
    W = torch.zeros(V, D, dtype=BF, device="cuda")
    t = torch.zeros(P, dtype=I32, device="cuda")
    old = (torch.rand(V, D, generator=g) * (P / V)).to(dtype).cuda()
    dW = old.clone()
    df2.unary_loss_grad(h, W, t, row_weights=w, dh=None, dW=dW, accumulate=accumulate)
    want = ((w.double() / V) @ h.double()).expand(V - 1, D)
    room = (256 + P / 4096 / 2 + 4) * 2.0 ** -23 * want
    if accumulate:
        want = want + old[1:].double()
        room = room + 2.0 ** -24 * want
    half = torch.finfo(dtype).eps / 2
    off = dW[1:].double() - want
    assert bool((off.abs() <= room * (1 + half) + half * want).all()), float((off / want).abs().max())
    # and not all to one side: the mean of many roundings, and of cuts as long as a piece's
    assert float((off / want).mean().abs()) <= 256 * 2.0 ** -23 + (0 if dtype == F32 else half)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("live", [900, 2500, 4096, 5000])
def test_rows_without_a_target_change_no_sum(df2, live, dtype):
    """The sums are those of the rows with a target alone, however many others there are."""
    P, V, D = 6000, 300, 136
    g = torch.Generator().manual_seed(live)
    h, W = torch.randn(P, D, generator=g).to(BF).cuda(), (torch.randn(V, D, generator=g) / 4).to(BF).cuda()
    some = torch.randperm(P, generator=g)[:live].sort().values.cuda()
    t = torch.full((P,), -1, dtype=I32, device="cuda")
    t[some] = torch.randint(0, V, (live,), generator=g).to(I32).cuda()
    a = df2.unary_loss_grad(h, W, t, dW=True, dtype=dtype)
    b = df2.unary_loss_grad(h[some], W, t[some], dW=True, dtype=dtype)
    assert torch.equal(a[3], b[3])
    assert torch.equal(a[0][some], b[0])


def test_replays_with_other_rows(df2):
    """A captured capped call of many rows, replayed with all of them, some and next to none live: the
    targets' slopes and the pieces of dW's sums are those of the rows of that replay."""
    P, V, D = 9000, 500, 72
    g = torch.Generator().manual_seed(6)
    h, W = torch.randn(P, D, generator=g).to(BF).cuda(), (torch.randn(V, D, generator=g) / 3).to(BF).cuda()
    ws = torch.empty(df2.unary_loss_grad_workspace_size(P, D, V, True, True), dtype=torch.uint8, device="cuda")
    t = torch.randint(0, V, (P,), generator=g).to(I32).cuda()
    dh, dW = torch.empty(P, D, device="cuda"), torch.empty(V, D, device="cuda")
    out = (torch.empty(P, device="cuda"), torch.empty(P, device="cuda"))
    df2.unary_loss_grad(h, W, t, final_logit_softcapping=2.0, dW=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        df2.unary_loss_grad(h, W, t, final_logit_softcapping=2.0, dh=dh, dW=dW, workspace=ws, out=out)
    every = t.clone()
    for masked in (0.0, 0.4, 0.6, 0.999, 0.0):
        t.copy_(torch.where(torch.rand(P, generator=g).cuda() < masked, torch.full_like(every, -1), every.roll(7)))
        h.copy_(h.roll(1, 0))
        ws.fill_(0xFF)  # nothing is left over from a replay before
        graph.replay()
        want = df2.unary_loss_grad(h, W, t, final_logit_softcapping=2.0, dW=True, dtype=F32)
        for a, b in zip((*out, dh, dW), want):
            assert torch.equal(a.nan_to_num(-1.0), b.nan_to_num(-1.0))
