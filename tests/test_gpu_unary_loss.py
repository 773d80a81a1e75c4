"""unary_ce and unary_loss_grad on the GPU against their definition in 64 bits, element by
element within what the roundings allow (unary_loss_ref)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from unary_loss_ref import check, reference  # noqa: E402

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
    w = torch.rand(P, generator=g) * 2
    return h.cuda(), W.cuda(), t.cuda(), w.cuda()


def compare(df2, h, W, t, w, mul=1.0, cap=0.0, dtype=BF, dW=True, accumulate=False, **more):
    keep = dW.clone() if isinstance(dW, torch.Tensor) else None
    want, room = reference(h, W, t, w, mul, cap, keep if accumulate else None)
    got = df2.unary_loss_grad(h, W, t, row_weights=w, output_multiplier=mul, final_logit_softcapping=cap, dtype=dtype,
                              dW=dW, accumulate=accumulate, **more)
    if accumulate:  # the old value, as it is held, is added in fp32
        room["dW"] = room["dW"] + 2.0 ** -24 * (want[3].abs() + keep.double().abs())
    worst = {n: check(n, a, b, room[n]) for n, a, b in zip(("loss", "lse", "dh", "dW"), got, want) if a is not None}
    loss, lse = df2.unary_ce(h, W, t, output_multiplier=mul, final_logit_softcapping=cap)
    assert torch.equal(loss.nan_to_num(-1.0), got[0].nan_to_num(-1.0))
    assert torch.equal(lse.nan_to_num(-1.0), got[1].nan_to_num(-1.0))
    return worst


SIZES = [(1, 1, 8), (1, 2, 8), (3, 5, 16), (8, 127, 64), (8, 1000, 72), (16, 4096, 256), (63, 129, 520), (64, 257, 64),
         (65, 255, 8), (130, 777, 1032), (256, 256, 512), (257, 513, 264), (300, 2050, 576), (600, 9001, 136),
         (5, 33001, 1024)]


@pytest.mark.parametrize("P, V, D", SIZES)
def test_sizes(df2, P, V, D):
    compare(df2, *inputs(P + V, P, V, D))


@pytest.mark.parametrize("mul, cap", [(1.0, 0.0), (0.8, 0.0), (1.0, 30.0), (0.5, 5.0), (3.0, 2.0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_maps_and_types(df2, mul, cap, dtype):
    compare(df2, *inputs(3, 140, 1500, 200), mul=mul, cap=cap, dtype=dtype)


@pytest.mark.parametrize("cap", [0.0, 8.0])
def test_gradients_against_differences(df2, cap):
    """Steps of 2^-6 in h and W that bf16 holds exactly.  Third order: by the 64-bit definition's
    own difference; the losses' error by their bounds; the gradient's by its."""
    g = torch.Generator().manual_seed(5)
    P, V, D = 24, 300, 64
    grid = lambda *s: torch.randint(-100, 101, s, generator=g).float() / 64  # noqa: E731
    h, W = grid(P, D).to(BF).cuda(), (grid(V, D) / 4).to(BF).cuda()
    t = torch.randint(0, V, (P,), generator=g).to(I32).cuda()
    dh_, dW_ = (torch.randint(-1, 2, x.shape, generator=g).float().cuda() / n for x, n in ((h, 64), (W, 256)))
    loss, lse, dh, dW = df2.unary_loss_grad(h, W, t, final_logit_softcapping=cap, dW=True, dtype=F32)
    (_, _, rh, rW), room = reference(h, W, t, cap=cap)
    for which, d, got, exact, bound in (("h", dh_, dh, rh, room["dh"]), ("W", dW_, dW, rW, room["dW"])):
        def moved(sign, f):
            a, b = (h + sign * d.to(BF), W) if which == "h" else (h, W + sign * d.to(BF))
            return f(a, b)
        gpu = [moved(s, lambda a, b: df2.unary_ce(a, b, t, final_logit_softcapping=cap)[0]).double() for s in (1, -1)]
        ref = [moved(s, lambda a, b: reference(a, b, t, cap=cap)) for s in (1, -1)]
        third = abs(float((ref[0][0][0] - ref[1][0][0]).sum() / 2 - (exact * d).sum()))
        losses = float((ref[0][1]["loss"] + ref[1][1]["loss"]).sum() / 2)
        grads = float((bound * d.abs()).sum()) + 2.0 ** -23 * float((exact * d).abs().sum())
        diff = float((gpu[0] - gpu[1]).sum() / 2) - float((got.double() * d.double()).sum())
        assert abs(diff) <= third + losses + grads, (which, diff, third, losses, grads)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P, V, D", [(40, 300, 72), (300, 1000, 1032), (70, 513, 8)])
def test_accumulate(df2, dtype, P, V, D):
    h, W, t, w = inputs(9, P, V, D)
    dW = torch.randn(V, D, generator=torch.Generator().manual_seed(1)).to(dtype).cuda() * 1e-2
    compare(df2, h, W, t, w, dW=dW, accumulate=True)


def test_which_gradients(df2):
    h, W, t, w = inputs(10, 100, 700, 128)
    loss, lse, dh, dW = df2.unary_loss_grad(h, W, t, row_weights=w, dW=True)
    a = df2.unary_loss_grad(h, W, t, row_weights=w)
    b = df2.unary_loss_grad(h, W, t, row_weights=w, dh=None, dW=True)
    c = df2.unary_loss_grad(h, W, t, dh=None)
    assert a[3] is None and b[2] is None and c[2] is None and c[3] is None
    assert torch.equal(a[2], dh) and torch.equal(b[3], dW)
    for x in (a, b, c):
        assert torch.equal(x[0].nan_to_num(-1), loss.nan_to_num(-1)) and torch.equal(x[1].nan_to_num(-1), lse.nan_to_num(-1))
    one = df2.unary_loss_grad(h, W, t, row_weights=torch.ones_like(w))[2]
    assert torch.equal(df2.unary_loss_grad(h, W, t)[2], one)
    out = (torch.empty(100, device="cuda"), None)
    mine = torch.full((100, 128), 9.0, device="cuda")
    got = df2.unary_loss_grad(h, W, t, row_weights=w, dh=mine, out=out)
    assert got[0] is out[0] and got[1] is None and got[2] is mine
    check("dh", mine, *(x[i] for x, i in zip(reference(h, W, t, w), (2, "dh"))))


def test_rows_without_a_target(df2):
    """Nothing of such a row is used: NaN, infinities and any weight leave no trace."""
    h, W, t, w = inputs(11, 130, 600, 200, masked=0.4)
    want = df2.unary_loss_grad(h, W, t, row_weights=w, dW=True)
    gone = t < 0
    for bad in (float("nan"), float("inf"), -float("inf")):
        h2, w2 = h.clone(), w.clone()
        h2[gone], w2[gone] = bad, bad
        got = df2.unary_loss_grad(h2, W, t, row_weights=w2, dW=True)
        for a, b in zip(got, want):
            assert torch.equal(a.nan_to_num(-1.0), b.nan_to_num(-1.0))
    assert bool(want[0][gone].isnan().all()) and not bool(want[0][~gone].isnan().any())
    assert not bool(want[2][gone].any())
    # none at all
    none = torch.full_like(t, -5)
    for dW0, accumulate in ((torch.full((600, 200), 7.0, device="cuda"), False),
                            (torch.full((600, 200), 7.0, device="cuda"), True)):
        loss, lse, dh, dW = df2.unary_loss_grad(h, W, none, dW=dW0, accumulate=accumulate)
        assert bool(loss.isnan().all()) and bool(lse.isnan().all()) and not bool(dh.any())
        assert bool((dW == (7.0 if accumulate else 0.0)).all())


def test_targets_out_of_range(df2):
    h, W, t, w = inputs(12, 50, 333, 64, masked=0.0)
    status = torch.zeros(1, dtype=I32, device="cuda")
    df2.unary_loss_grad(h, W, t, dev_status=status)
    assert int(status) == 0
    t2, t3 = t.clone(), t.clone()
    t2[7], t2[20] = 333, 2 ** 31 - 1
    t3[7], t3[20] = -1, -2 ** 31
    a = df2.unary_loss_grad(h, W, t2, dW=True, dev_status=status)
    assert int(status) == df2.DF2_STATUS_ID_OUT_OF_RANGE
    for x, y in zip(a, df2.unary_loss_grad(h, W, t3, dW=True)):
        assert torch.equal(x.nan_to_num(-1.0), y.nan_to_num(-1.0))
    status.zero_()
    df2.unary_ce(h, W, t2, dev_status=status)
    assert int(status) == df2.DF2_STATUS_ID_OUT_OF_RANGE


def test_nan_reaches_its_own_row(df2):
    h, W, t, w = inputs(13, 60, 400, 64, masked=0.1)
    t[3] = 5
    h[3, 10] = float("nan")
    loss, lse, dh, dW = df2.unary_loss_grad(h, W, t, row_weights=w, dW=True)
    live = t >= 0
    assert torch.equal(loss.isnan(), ~live | (torch.arange(60, device="cuda") == 3)) and bool(lse[3].isnan())
    assert bool(dh[3].isnan().all()) and not bool(dh[live & (torch.arange(60, device="cuda") != 3)].isnan().any())
    assert bool(dW.isnan().all())  # every row of dW is a sum with that row's part
    keep = torch.arange(60, device="cuda") != 3
    want = df2.unary_loss_grad(h[keep].contiguous(), W, t[keep].contiguous(), row_weights=w[keep].contiguous())
    assert torch.equal(loss[keep].nan_to_num(-1), want[0].nan_to_num(-1)) and torch.equal(dh[keep], want[2])


def test_extreme_logits(df2):
    """All but certain, all but impossible, all equal, and spreads far beyond exp's range."""
    g = torch.Generator().manual_seed(14)
    D, V = 64, 777
    W = torch.randn(V, D, generator=g).to(BF)
    h = torch.randn(8, D, generator=g).to(BF)
    t = torch.arange(8) * 90
    h[0] = 4 * W[t[0]]                      # the target far ahead: loss near 0
    h[1] = -4 * W[t[1]]                     # far behind
    h[2] = 0.0                              # all equal: log V
    h[3] = 60 * W[t[3]]                     # logits of thousands
    h[4] = -60 * W[t[4]]
    h[5] = 2.0 ** -60 * h[5].float()        # logits near 2^-57
    h, W, t = h.cuda(), W.cuda(), t.to(I32).cuda()
    w = torch.ones(8, device="cuda")
    compare(df2, h, W, t, w)
    compare(df2, h, W, t, w, cap=20.0)
    loss = df2.unary_ce(h, W, t)[0]
    assert 0.0 <= float(loss[0]) < 1e-12 and abs(float(loss[2]) - 6.655440350367647) < 2e-6


def test_weights_of_any_sign(df2):
    h, W, t, w = inputs(15, 90, 500, 96)
    w = w - 1.0
    w[::7] = 0.0
    compare(df2, h, W, t, w)
    got = df2.unary_loss_grad(h, W, t, row_weights=w)[2]
    assert not bool(got[w == 0.0].any())


def test_equal_inputs_give_equal_bits(df2):
    h, W, t, w = inputs(16, 500, 5000, 520)
    a, b = (df2.unary_loss_grad(h, W, t, row_weights=w, dW=True, dtype=F32) for _ in range(2))
    for x, y in zip(a, b):
        assert torch.equal(x.nan_to_num(-1.0), y.nan_to_num(-1.0))


def test_where_rows_lie_does_not_matter(df2):
    """The rows with a target give the same bits alone as among others without one."""
    h, W, t, w = inputs(17, 200, 900, 128, masked=0.5)
    live = t >= 0
    a = df2.unary_loss_grad(h, W, t, row_weights=w, dW=True)
    b = df2.unary_loss_grad(h[live].contiguous(), W, t[live].contiguous(), row_weights=w[live].contiguous(), dW=True)
    assert torch.equal(a[0][live], b[0]) and torch.equal(a[2][live], b[2]) and torch.equal(a[3], b[3])


def test_more_than_one_piece(df2):
    """2^22 columns: 700 rows go in two pieces (of 512), with all rows live, with the second
    piece empty, and added to what dW holds; the definition's sums a few rows at a time."""
    V, D, P = 1 << 22, 16, 700
    for masked, dtype, accumulate in ((0.0, BF, False), (0.5, F32, False), (0.0, BF, True)):
        h, W, t, w = inputs(18, P, V, D, masked=masked)
        if masked:
            assert int((t >= 0).sum()) < 512
        dW = torch.ones(V, D, dtype=dtype, device="cuda") * 2.0 ** -10
        keep = dW.double() if accumulate else torch.zeros(V, D, dtype=torch.float64, device="cuda")
        room_W = torch.zeros(V, D, dtype=torch.float64, device="cuda")
        got = df2.unary_loss_grad(h, W, t, row_weights=w, dW=dW, accumulate=accumulate)
        for some in torch.arange(P, device="cuda").split(50):
            want, room = reference(h[some], W, t[some], w[some])
            for n, i in (("loss", 0), ("lse", 1), ("dh", 2)):
                check(n, got[i][some], want[i], room[n])
            keep += want[3]
            room_W += room["dW"]
        check("dW", got[3], keep, room_W + 2.0 ** -22 * keep.abs() + (2.0 ** -24 * 2.0 ** -10 if accumulate else 0.0))
        torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("P, V, D", [(1600, 900, 2568), (2100, 600, 136)])
def test_many_tiles_and_long_sums(df2, P, V, D, dtype):
    """dh of more tiles than clusters, some whole and some cut, an odd number of them each way; dW's
    sums of over 2,048 rows, stored and added."""
    h, W, t, w = inputs(21, P, V, D, masked=0.02)
    compare(df2, h, W, t, w, dtype=dtype)
    dW = (torch.randn(V, D, generator=torch.Generator().manual_seed(2)) * 1e-2).to(dtype).cuda()
    compare(df2, h, W, t, w, dtype=dtype, dW=dW, accumulate=True)


def test_loss_alone_in_pieces(df2):
    """2^24 columns: the statistics of 700 rows go in two pieces; each row is as it is by itself, and
    some are as the definition says."""
    V, D, P = 1 << 24, 8, 700
    h, W, t, w = inputs(22, P, V, D, masked=0.1)
    loss, lse = df2.unary_ce(h, W, t)
    for some in (slice(0, 300), slice(300, 555), slice(555, 700)):
        a, b = df2.unary_ce(h[some], W, t[some])
        assert torch.equal(a.nan_to_num(-1.0), loss[some].nan_to_num(-1.0))
        assert torch.equal(b.nan_to_num(-1.0), lse[some].nan_to_num(-1.0))
    rows = torch.tensor([0, 255, 511, 512, 699], device="cuda")
    x = h[rows].double() @ W.double().T
    want = torch.logsumexp(x, 1)
    live = t[rows] >= 0
    # five steps of at most 2^-23 of the sum of a logit's terms, exponents, and sums of 2^18 values
    room = 5 * 2.0 ** -23 * float((h[rows].double().abs().sum(1) * W.double().abs().max()).max()) + 2.0 ** -16
    assert bool(((lse[rows] - want).abs()[live] <= room).all())
    assert bool(((loss[rows] - (want - x.gather(1, t[rows].clamp(min=0).long()[:, None])[:, 0])).abs()[live] <= 2 * room).all())


def test_two_host_threads(df2):
    """Calls from two threads on streams of their own, their shapes taking other kernels."""
    import threading
    a, b = inputs(34, 700, 3000, 512), inputs(35, 60, 5000, 1032)
    want = [df2.unary_loss_grad(*s[:3], row_weights=s[3], dW=True, final_logit_softcapping=c) for s, c in ((a, 0.0), (b, 20.0))]
    torch.cuda.synchronize()
    wrong = []

    def work(s, cap, expected):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got = df2.unary_loss_grad(*s[:3], row_weights=s[3], dW=True, final_logit_softcapping=cap)
                stream.synchronize()
                wrong.extend(not torch.equal(x.nan_to_num(-1.0), y.nan_to_num(-1.0)) for x, y in zip(got, expected))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(s, c, e)) for s, c, e in ((a, 0.0, want[0]), (b, 20.0, want[1]))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert len(wrong) == 160 and not any(wrong)


def test_offsets_past_32_bits(df2):
    """A head of 2.46e9 elements: logits, dh and the ends of dW, in fp32 and added in bf16, against sums in
    64 bits a piece of the head at a time."""
    V, D, P = 600_000, 4096, 8
    g = torch.Generator(device="cuda").manual_seed(40)
    W = torch.empty(V, D, dtype=BF, device="cuda").normal_(0.0, 0.04, generator=g)
    h = torch.randn(P, D, generator=g, device="cuda").to(BF)
    t = torch.tensor([0, 1, 299_999, 524_288, 599_998, 599_999, -1, 400_000], dtype=I32, device="cuda")
    live = t >= 0
    x, S = [], []
    for w in W.split(50_000):
        x.append(h.double() @ w.double().T)
        S.append(h.double().abs() @ w.double().abs().T)
    x, du = torch.cat(x, 1), (D / 16 + 4) * 2.0 ** -23 * torch.cat(S, 1)
    lse = torch.logsumexp(x, 1)
    gr = torch.exp(x - lse[:, None])
    gr[torch.arange(P, device="cuda"), t.long().clamp(min=0)] -= 1.0
    gr[~live] = 0.0
    # a factor: its logit's and the log-sum-exp's errors, exp's and the sums', fp16 and bf16
    dg = gr.abs() * (2 * du.amax(1, keepdim=True) + 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15) + 2.0 ** -36
    want, room = torch.zeros(P, D, dtype=torch.float64, device="cuda"), torch.zeros(P, D, dtype=torch.float64, device="cuda")
    for k, w in enumerate(W.split(50_000)):
        part = slice(50_000 * k, 50_000 * k + len(w))
        want += gr[:, part] @ w.double()
        room += (dg[:, part] + (V / 16 + 4) * 2.0 ** -23 * gr[:, part].abs()) @ w.double().abs()
    rows = torch.cat([torch.arange(0, 64), torch.arange(299_990, 300_010), torch.arange(524_280, 524_300),
                      torch.arange(V - 64, V)]).cuda()
    wW, rW = gr[:, rows].T @ h.double(), dg[:, rows].T @ h.double().abs()
    dW = torch.full((V, D), 0.5, dtype=BF, device="cuda")
    for more in (dict(dW=True, dtype=F32), dict(dW=dW, accumulate=True)):
        loss, l, dh, got = df2.unary_loss_grad(h, W, t, **more)
        assert bool(((l - lse).abs()[live] <= du.amax(1)[live] + 2.0 ** -17).all()) and bool(l[~live].isnan().all())
        xt = x[torch.arange(P, device="cuda"), t.long().clamp(min=0)]
        assert bool(((loss - (lse - xt)).abs()[live] <= 2 * du.amax(1)[live] + 2.0 ** -17).all())
        check("dh", dh, want, room)
        had = 0.5 if "accumulate" in more else 0.0
        check("dW", got[rows], wW + had, rW + 2.0 ** -22 * (wW.abs() + had))
        del got
        torch.cuda.empty_cache()


def test_zero_rows(df2):
    h, W, t, w = inputs(19, 4, 100, 64)
    loss, lse, dh, dW = df2.unary_loss_grad(h[:0], W, t[:0], dW=torch.ones(100, 64, device="cuda"))
    assert loss.shape == (0,) and dh.shape == (0, 64) and not bool(dW.any())
    dW = torch.ones(100, 64, device="cuda")
    df2.unary_loss_grad(h[:0], W, t[:0], dW=dW, accumulate=True)
    assert bool((dW == 1).all())
    assert df2.unary_ce(h[:0], W, t[:0])[0].shape == (0,)


def test_graph(df2):
    """A captured call, replayed on other inputs with other rows live; two graphs that share a
    workspace, replayed one after the other."""
    P, V, D = 300, 3000, 256
    sets = [inputs(20 + k, P, V, D, masked=m) for k, m in enumerate((0.0, 0.3, 0.97))]
    h, W, t, w = (x.clone() for x in sets[0])
    ws = torch.empty(df2.unary_loss_grad_workspace_size(P, D, V, True, True), dtype=torch.uint8, device="cuda")
    dh, dW = torch.empty(P, D, dtype=BF, device="cuda"), torch.empty(V, D, dtype=BF, device="cuda")
    out = (torch.empty(P, device="cuda"), torch.empty(P, device="cuda"))
    out2 = (torch.empty(P, device="cuda"), torch.empty(P, device="cuda"))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        df2.unary_loss_grad(h, W, t, row_weights=w, dh=dh, dW=dW, workspace=ws, out=out)
    with torch.cuda.graph(graphs[1]):
        df2.unary_ce(h, W, t, workspace=ws, out=out2)
    for s in sets:
        for a, b in zip((h, W, t, w), s):
            a.copy_(b)
        graphs[0].replay()
        graphs[1].replay()
        want = df2.unary_loss_grad(*s[:3], row_weights=s[3], dW=True)
        for a, b in zip((*out, dh, dW, *out2), (*want, *want[:2])):
            assert torch.equal(a.nan_to_num(-1.0), b.nan_to_num(-1.0))


def test_two_streams_at_once(df2):
    """Calls on two streams, their own workspaces, again and again."""
    a, b = inputs(30, 520, 4000, 512), inputs(31, 100, 9000, 256)
    want = [df2.unary_loss_grad(*s[:3], row_weights=s[3], dW=True) for s in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for k, s in enumerate((a, b)):
            got[k].append(df2.unary_loss_grad(*s[:3], row_weights=s[3], dW=True, stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        for g in got[k]:
            for x, y in zip(g, want[k]):
                assert torch.equal(x.nan_to_num(-1.0), y.nan_to_num(-1.0))


def test_the_logits_are_unary_topks(df2):
    """The loss of a row is lse - its target's logit: with the top candidate as the target, the
    logit that unary_topk gives."""
    h, W, t, w = inputs(32, 64, 3000, 256, masked=0.0)
    for mul, cap in ((1.0, 0.0), (0.7, 30.0)):
        ids, vals, _ = df2.unary_topk(h, W, 4, output_multiplier=mul, final_logit_softcapping=cap)
        for k in (0, 3):
            loss, lse = df2.unary_ce(h, W, ids[:, k].contiguous(), output_multiplier=mul, final_logit_softcapping=cap)
            du = (256 / 16 + 4) * 2.0 ** -23 * (h.double().abs() @ W.double().abs().T).amax(1)
            room = 3 * du + 2.0 ** -20 * (lse.abs() + vals[:, k].abs()) + 2.0 ** -18
            assert bool(((lse - loss - vals[:, k]).abs() <= room).all())


def test_refusals_on_the_device(df2):
    h, W, t, w = inputs(33, 16, 100, 64)
    with pytest.raises(df2.DFlash2Error):
        df2.unary_loss_grad(h, W, t, dh=h)  # over an input
    both = torch.empty(100, 64, dtype=BF, device="cuda")
    with pytest.raises(df2.DFlash2Error):
        df2.unary_loss_grad(h, W, t, dh=both[:16], dW=both)
    with pytest.raises(ValueError):
        df2.unary_loss_grad(h, W, t, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(df2.DFlash2Error):
        df2.unary_ce(h, W, t, output_multiplier=0.0)
    with pytest.raises(df2.DFlash2Error):
        df2.unary_ce(h[:, :60].contiguous(), W[:, :60].contiguous(), t)
